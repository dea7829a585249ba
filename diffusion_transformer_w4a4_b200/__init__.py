"""Python binding of libsvdq, the SVDQuant W4A4 linear layer (svdq_w4a4) for one
NVIDIA B200 (sm_100a).

Argument marshalling only: every step of the layer runs in the CUDA library
(include/svdq.h).  torch is used for device memory and streams.  There is no
CPU fallback: if libsvdq.so is missing or cannot be loaded, every call raises.

Entry points keep the C names (svdq_prepare, svdq_pack, svdq_layer_create,
svdq_forward, ..., svdq_awq_* for the awq_w4a16 layer, svdq_w8a8_* and svdq_fp8_*
for the 8-bit layers).  `SvdqLinear`, `AwqLinear`, `W8A8Linear` and `Fp8Linear`
bundle them for nn.Linear-style use.  svdq_qk_norm_rope and svdq_cross_attn, the
steps between a block's projections, take torch tensors [batch, tokens, heads, dim].
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# SVDQ_LIBRARY=debug selects the bounds-checked debug variant (libsvdq_debug.so,
# built by build.build(debug=True)); the default is the release library.
LIB_PATH = os.path.join(_HERE, "libsvdq_debug.so" if os.environ.get("SVDQ_LIBRARY") == "debug" else "libsvdq.so")

SVDQ_OK = 0
SVDQ_ERR_INVALID_ARG = 1
SVDQ_ERR_UNSUPPORTED_DEVICE = 2
SVDQ_ERR_OOM = 3
SVDQ_ERR_CUDA = 4
SVDQ_ERR_NUMERIC = 5
SVDQ_ERR_TIMEOUT = 6
SVDQ_ERR_BOUNDS = 7
SVDQ_INT4_G64 = 1
SVDQ_NVFP4_G16 = 2
FORMATS = {"int4": SVDQ_INT4_G64, "nvfp4": SVDQ_NVFP4_G16, SVDQ_INT4_G64: SVDQ_INT4_G64,
           SVDQ_NVFP4_G16: SVDQ_NVFP4_G16}


def _fmt(f) -> int:
    """Format name or code -> code (unknown integers pass through for the library to reject)."""
    return int(f) if isinstance(f, (int, np.integer)) else FORMATS[f]


class SvdqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {svdq_status_string(status)}")


class svdq_canonical(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("rank", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("g_x", ctypes.c_float), ("g_w", ctypes.c_float),
                ("reserved", ctypes.c_float), ("lambda_", ctypes.c_void_p), ("inv_lambda", ctypes.c_void_p),
                ("L1", ctypes.c_void_p), ("L2", ctypes.c_void_p), ("wcodes", ctypes.c_void_p),
                ("wscales", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class svdq_awq_canonical(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("alpha", ctypes.c_float), ("reserved", ctypes.c_float),
                ("s", ctypes.c_void_p), ("inv_s", ctypes.c_void_p), ("wcodes", ctypes.c_void_p),
                ("wscales", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


_lib = None
_EXPORTS = {
    # name: (restype, argtypes)
    "svdq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "svdq_abi_version": (ctypes.c_int, []),
    "svdq_debug_build": (ctypes.c_int, []),
    "svdq_canonical_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                            ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_prepare": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                    ctypes.POINTER(svdq_canonical)]),
    "svdq_packed_size": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_pack": (ctypes.c_int, [ctypes.POINTER(svdq_canonical), ctypes.c_void_p, ctypes.c_size_t]),
    "svdq_device_check": (ctypes.c_int, [ctypes.c_int]),
    "svdq_layer_create": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                         ctypes.POINTER(ctypes.c_void_p)]),
    "svdq_layer_destroy": (None, [ctypes.c_void_p]),
    "svdq_workspace_size": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_workspace_layout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t),
                                             ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_workspace_init": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p]),
    "svdq_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_quantize_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_int4_group_acc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p, ctypes.c_void_p]),
    "svdq_read_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.POINTER(ctypes.c_int)]),
    "svdq_set_wait_limit": (ctypes.c_int, [ctypes.c_uint64]),
    "svdq_forward_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "svdq_mlp_fusable": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "svdq_gemm_gelu_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                               ctypes.c_size_t, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "svdq_mlp_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_awq_canonical_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_awq_prepare": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(svdq_awq_canonical)]),
    "svdq_awq_packed_size": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_awq_pack": (ctypes.c_int, [ctypes.POINTER(svdq_awq_canonical), ctypes.c_void_p, ctypes.c_size_t]),
    "svdq_awq_layer_create": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.POINTER(ctypes.c_void_p)]),
    "svdq_awq_layer_destroy": (None, [ctypes.c_void_p]),
    "svdq_awq_read_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "svdq_awq_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "svdq_w8a8_prepare": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.POINTER(ctypes.c_float)]),
    "svdq_w8a8_packed_size": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_w8a8_pack": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_size_t]),
    "svdq_w8a8_layer_create": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int64,
                                              ctypes.c_float, ctypes.POINTER(ctypes.c_void_p)]),
    "svdq_w8a8_layer_destroy": (None, [ctypes.c_void_p]),
    "svdq_w8a8_workspace_size": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_w8a8_quantize_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                              ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_w8a8_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_w8a8_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_fp8_prepare": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "svdq_fp8_packed_size": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_fp8_pack": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t]),
    "svdq_fp8_layer_create": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.POINTER(ctypes.c_void_p)]),
    "svdq_fp8_layer_destroy": (None, [ctypes.c_void_p]),
    "svdq_fp8_workspace_size": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "svdq_fp8_quantize_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                             ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_fp8_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_fp8_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svdq_fp8_read_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.POINTER(ctypes.c_int)]),
    # (svdq_qk_norm_rope and svdq_cross_attn below go through _marshal.so, by the functions' addresses; called by these
    # types they take the structures svdq_norm_rope_args and svdq_attn_args as packed bytes)
    "svdq_qk_norm_rope": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_char_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]),
    "svdq_cross_attn": (ctypes.c_int, [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_void_p]),
    "svdq_w8a8_read_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                             ctypes.POINTER(ctypes.c_int)]),
}


def lib() -> ctypes.CDLL:
    """The loaded libsvdq.so; raises if it was not built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{os.path.basename(LIB_PATH)} not found at {LIB_PATH}: build it with "
                               "`python -m diffusion_transformer_w4a4_b200.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != SVDQ_OK:
        raise SvdqError(status, where)


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        assert a.flags["C_CONTIGUOUS"]
        return a.ctypes.data
    return a.data_ptr()  # torch tensor


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    return int(getattr(stream, "cuda_stream", stream))


def _stream_context(stream, device):
    """`stream` (a torch stream, or a raw handle of one of `device`) as the current stream of `device`."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))  # 0: the default stream (ExternalStream(0) is a new one)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"a stream of {stream.device} for work on {device}")
    return torch.cuda.stream(stream)


def _current_handle(device) -> int:
    """The handle of the device's current stream (torch's Python stream objects take microseconds)."""
    return (_calls_module or _calls()).current_stream(device.index)


def _on(stream, device):
    """The stream that a call works on as the current one, for a call that allocates: what it makes is that stream's memory.
    (Making a stream current costs the host 8 us; None leaves the current one.)"""
    return contextlib.nullcontext() if stream is None else _stream_context(stream, device)


def _empty_like(x, stream):
    """An output like x, of the memory of the stream that will write it."""
    if stream is None or not x.is_cuda:  # (a tensor of the host is refused later, with the others' checks)
        return _torch().empty_like(x)
    with _stream_context(stream, x.device):
        return _torch().empty_like(x)


_torch_module = None


def _torch():
    """torch, imported at the first use (this module loads without it)."""
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


# ----------------------------------------------------------------------------- C names
def svdq_status_string(status: int) -> str:
    return lib().svdq_status_string(int(status)).decode()


def svdq_debug_build() -> int:
    """1 when the loaded library is the bounds-checked debug variant."""
    return int(lib().svdq_debug_build())


def svdq_abi_version() -> int:
    return int(lib().svdq_abi_version())


def svdq_canonical_sizes(N: int, K: int, rank: int, fmt) -> list[int]:
    sizes = (ctypes.c_size_t * 7)()
    _check(lib().svdq_canonical_sizes(N, K, rank, _fmt(fmt), sizes), "svdq_canonical_sizes")
    return list(sizes)


def _canonical_arrays(N, K, rank, fmt):
    fmt = _fmt(fmt)
    return dict(
        N=N, K=K, rank=rank, fmt=fmt,
        lambda_=np.zeros(K, np.float32), inv_lambda=np.zeros(K, np.float32),
        L1=np.zeros((K, rank), np.uint16), L2=np.zeros((rank, N), np.uint16),
        wcodes=np.zeros((N, K // 2), np.uint8),
        wscales=np.zeros((N, K // 64), np.uint16) if fmt == SVDQ_INT4_G64 else np.zeros((N, K // 16), np.uint8),
        bias=np.zeros(N, np.uint16), g_x=1.0, g_w=1.0, alpha=0.5)


def _to_struct(c: dict) -> svdq_canonical:
    s = svdq_canonical()
    s.N, s.K, s.rank, s.fmt = int(c["N"]), int(c["K"]), int(c["rank"]), _fmt(c["fmt"])
    s.alpha, s.g_x, s.g_w = float(c.get("alpha", 0.5)), float(c.get("g_x", 1.0)), float(c.get("g_w", 1.0))
    for f in ("lambda_", "inv_lambda", "L1", "L2", "wcodes", "wscales", "bias"):
        arr = c.get(f)
        setattr(s, f, None if arr is None or arr.size == 0 else arr.ctypes.data)
    return s


def svdq_prepare(W: np.ndarray, bias, act_absmax: np.ndarray, alpha: float, rank: int, fmt) -> dict:
    """Host-side preparation (smoothing, truncated SVD, residual quantize).
    W: bf16 bits [N,K] uint16; bias: bf16 bits [N] or None; act_absmax: float32 [K]."""
    W = np.ascontiguousarray(W, np.uint16)
    N, K = W.shape
    c = _canonical_arrays(N, K, rank, fmt)
    s = _to_struct(c)
    b = None if bias is None else np.ascontiguousarray(bias, np.uint16)
    am = np.ascontiguousarray(act_absmax, np.float32)
    _check(lib().svdq_prepare(W.ctypes.data, None if b is None else b.ctypes.data, am.ctypes.data,
                              float(alpha), ctypes.byref(s)), "svdq_prepare")
    c["g_x"], c["g_w"], c["alpha"] = float(s.g_x), float(s.g_w), float(s.alpha)
    return c


def svdq_packed_size(N: int, K: int, rank: int, fmt) -> int:
    n = ctypes.c_size_t()
    _check(lib().svdq_packed_size(N, K, rank, _fmt(fmt), ctypes.byref(n)), "svdq_packed_size")
    return n.value


def svdq_pack(c: dict) -> np.ndarray:
    """Canonical prepared weights (dict of host arrays) -> device-layout blob (host bytes)."""
    c = dict(c)
    for f, dt in (("lambda_", np.float32), ("inv_lambda", np.float32), ("L1", np.uint16), ("L2", np.uint16),
                  ("wcodes", np.uint8), ("bias", np.uint16)):
        if c.get(f) is not None:
            c[f] = np.ascontiguousarray(c[f], dt)
    c["wscales"] = np.ascontiguousarray(c["wscales"])
    size = svdq_packed_size(c["N"], c["K"], c["rank"], c["fmt"])
    blob = np.zeros(size, np.uint8)
    s = _to_struct(c)
    _check(lib().svdq_pack(ctypes.byref(s), blob.ctypes.data, size), "svdq_pack")
    return blob


def svdq_device_check(device: int = 0) -> int:
    return int(lib().svdq_device_check(int(device)))


def svdq_layer_create(dev_blob, blob_bytes: int, N: int, K: int, rank: int, fmt, g_x: float, g_w: float):
    h = ctypes.c_void_p()
    _check(lib().svdq_layer_create(_ptr(dev_blob), blob_bytes, N, K, rank, _fmt(fmt), float(g_x), float(g_w),
                                   ctypes.byref(h)), "svdq_layer_create")
    return h


def svdq_layer_destroy(h) -> None:
    lib().svdq_layer_destroy(h)


def svdq_workspace_size(h, M: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().svdq_workspace_size(h, M, ctypes.byref(n)), "svdq_workspace_size")
    return n.value


def svdq_workspace_layout(h, M: int):
    off = (ctypes.c_size_t * 4)()
    sz = (ctypes.c_size_t * 4)()
    _check(lib().svdq_workspace_layout(h, M, off, sz), "svdq_workspace_layout")
    return list(off), list(sz)


def svdq_workspace_init(h, M: int, ws, stream=None) -> None:
    _check(lib().svdq_workspace_init(h, M, _ptr(ws), ws.numel(), _stream(stream)), "svdq_workspace_init")


def svdq_forward(h, X, M: int, Y, ws, stream=None) -> None:
    _check(lib().svdq_forward(h, _ptr(X), M, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)), "svdq_forward")


def svdq_quantize_act(h, X, M: int, ws, stream=None) -> None:
    _check(lib().svdq_quantize_act(h, _ptr(X), M, _ptr(ws), ws.numel(), _stream(stream)), "svdq_quantize_act")


def svdq_gemm(h, M: int, Y, ws, stream=None) -> None:
    _check(lib().svdq_gemm(h, M, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)), "svdq_gemm")


def svdq_int4_group_acc(h, M: int, ws, acc, stream=None) -> None:
    _check(lib().svdq_int4_group_acc(h, M, _ptr(ws), ws.numel(), _ptr(acc), _stream(stream)), "svdq_int4_group_acc")


def svdq_read_status(h, M: int, ws) -> int:
    """Status word of a caller workspace, or (ws=None) of the last
    svdq_forward_noalloc call for M tokens on the current device."""
    v = ctypes.c_int()
    nbytes = ws.numel() if ws is not None else 0
    _check(lib().svdq_read_status(h, M, _ptr(ws), nbytes, ctypes.byref(v)), "svdq_read_status")
    return int(v.value)


def svdq_forward_noalloc(h, X, M: int, Y, stream=None) -> None:
    """Forward without a caller workspace (library-owned 32 MiB scratch per GPU)."""
    _check(lib().svdq_forward_noalloc(h, _ptr(X), M, _ptr(Y), _stream(stream)), "svdq_forward_noalloc")


def svdq_mlp_fusable(up, down) -> int:
    """SVDQ_OK when the pair (up, down) can run as one fused MLP (see svdq_mlp_forward)."""
    return int(lib().svdq_mlp_fusable(up, down))


def svdq_gemm_gelu_quantize(up, down, M: int, ws_up, ws_dn, H=None, stream=None) -> None:
    """The up layer's GEMM with GELU and the down layer's quantizer in its epilogue."""
    _check(lib().svdq_gemm_gelu_quantize(up, down, M, _ptr(ws_up), ws_up.numel(), _ptr(ws_dn), ws_dn.numel(),
                                         _ptr(H), _stream(stream)), "svdq_gemm_gelu_quantize")


def svdq_mlp_forward(up, down, X, M: int, Y, ws_up, ws_dn, stream=None) -> None:
    """Y = down(GELU(up(X))) with the cross-layer fused GEMM in the middle."""
    _check(lib().svdq_mlp_forward(up, down, _ptr(X), M, _ptr(Y), _ptr(ws_up), ws_up.numel(), _ptr(ws_dn),
                                  ws_dn.numel(), _stream(stream)), "svdq_mlp_forward")


def svdq_set_wait_limit(cycles: int) -> None:
    _check(lib().svdq_set_wait_limit(int(cycles)), "svdq_set_wait_limit")


# ----------------------------------------------------------------------------- convenience
def _layer_device(device):
    """The CUDA device a layer lives on, always with its index."""
    import torch

    d = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    if d.type != "cuda":
        raise ValueError(f"a layer lives on a CUDA device, not {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


def _check_input(x, K: int, device):
    import torch

    if not (x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous() and x.shape[-1] == K):
        raise ValueError(f"expected a contiguous bf16 CUDA tensor [..., {K}], got {x.dtype} {tuple(x.shape)}")
    if x.device != device:
        raise ValueError(f"input on {x.device}, layer on {device}")


class SvdqLinear:
    """One svdq_w4a4 layer resident on `device` (default: the current CUDA device).

    Built from canonical prepared weights (svdq_prepare output, or any dict with
    the same arrays); `forward(x)` takes a bf16 CUDA tensor [M, K] on that device
    and returns bf16 [M, N].  Workspaces are cached per token count.  The handle
    is created, and every call that enqueues work is made, with the layer's
    device current (the library refuses a call from another device)."""

    def __init__(self, canonical: dict, device=None):
        import torch

        self.N, self.K, self.rank = int(canonical["N"]), int(canonical["K"]), int(canonical["rank"])
        self.fmt = _fmt(canonical["fmt"])
        self.g_x, self.g_w = float(canonical.get("g_x", 1.0)), float(canonical.get("g_w", 1.0))
        self.device = _layer_device(device)
        blob = svdq_pack(canonical)
        self.blob = torch.from_numpy(blob).to(self.device)
        with torch.cuda.device(self.device):
            self.handle = svdq_layer_create(self.blob, self.blob.numel(), self.N, self.K, self.rank, self.fmt,
                                            self.g_x, self.g_w)
        self._ws = {}

    def workspace(self, M: int):
        import torch

        ws = self._ws.get(M)
        if ws is None:
            ws = torch.empty(max(svdq_workspace_size(self.handle, M), 1024), dtype=torch.uint8, device=self.device)
            with torch.cuda.device(self.device):
                svdq_workspace_init(self.handle, M, ws)
            self._ws[M] = ws
        return ws

    def forward(self, x, out=None, stream=None):
        import torch

        _check_input(x, self.K, self.device)
        M = x.numel() // self.K
        with torch.cuda.device(self.device), _on(stream if out is None or M not in self._ws else None, self.device):
            y = out if out is not None else torch.empty(M, self.N, dtype=torch.bfloat16, device=x.device)
            svdq_forward(self.handle, x, M, y, self.workspace(M), stream)
        return y

    __call__ = forward

    def status(self, M: int) -> int:
        return svdq_read_status(self.handle, M, self.workspace(M))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.svdq_layer_destroy(h)
            self.handle = None


# ----------------------------------------------------------------------------- awq_w4a16
def svdq_awq_canonical_sizes(N: int, K: int) -> list[int]:
    sizes = (ctypes.c_size_t * 5)()
    _check(lib().svdq_awq_canonical_sizes(N, K, sizes), "svdq_awq_canonical_sizes")
    return list(sizes)


def _awq_arrays(N, K):
    return dict(N=N, K=K, alpha=0.0, s=np.zeros(K, np.float32), inv_s=np.zeros(K, np.float32),
                wcodes=np.zeros((N, K // 2), np.uint8), wscales=np.zeros((N, K // 64), np.uint16),
                bias=np.zeros(N, np.uint16))


def _awq_struct(c: dict) -> svdq_awq_canonical:
    st = svdq_awq_canonical()
    st.N, st.K, st.alpha = int(c["N"]), int(c["K"]), float(c.get("alpha", 0.0))
    for f in ("s", "inv_s", "wcodes", "wscales", "bias"):
        arr = c.get(f)
        setattr(st, f, None if arr is None else arr.ctypes.data)
    return st


def svdq_awq_prepare(W: np.ndarray, bias, X_calib: np.ndarray) -> dict:
    """Host-side activation-aware preparation of an awq_w4a16 layer.
    W: bf16 bits [N,K]; bias: bf16 bits [N] or None; X_calib: bf16 bits [M_calib, K]."""
    W = np.ascontiguousarray(W, np.uint16)
    X = np.ascontiguousarray(X_calib, np.uint16)
    N, K = W.shape
    c = _awq_arrays(N, K)
    st = _awq_struct(c)
    b = None if bias is None else np.ascontiguousarray(bias, np.uint16)
    _check(lib().svdq_awq_prepare(W.ctypes.data, None if b is None else b.ctypes.data, X.ctypes.data, X.shape[0],
                                  ctypes.byref(st)), "svdq_awq_prepare")
    c["alpha"] = float(st.alpha)
    return c


def svdq_awq_packed_size(N: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().svdq_awq_packed_size(N, K, ctypes.byref(n)), "svdq_awq_packed_size")
    return n.value


def svdq_awq_pack(c: dict) -> np.ndarray:
    c = dict(c)
    for f, dt in (("s", np.float32), ("inv_s", np.float32), ("wcodes", np.uint8), ("wscales", np.uint16),
                  ("bias", np.uint16)):
        if c.get(f) is not None:
            c[f] = np.ascontiguousarray(c[f], dt)
    size = svdq_awq_packed_size(c["N"], c["K"])
    blob = np.zeros(size, np.uint8)
    _check(lib().svdq_awq_pack(ctypes.byref(_awq_struct(c)), blob.ctypes.data, size), "svdq_awq_pack")
    return blob


def svdq_awq_layer_create(dev_blob, blob_bytes: int, N: int, K: int):
    h = ctypes.c_void_p()
    _check(lib().svdq_awq_layer_create(_ptr(dev_blob), blob_bytes, N, K, ctypes.byref(h)), "svdq_awq_layer_create")
    return h


def svdq_awq_layer_destroy(h) -> None:
    lib().svdq_awq_layer_destroy(h)


def svdq_awq_read_status(h) -> int:
    v = ctypes.c_int()
    _check(lib().svdq_awq_read_status(h, ctypes.byref(v)), "svdq_awq_read_status")
    return v.value


def svdq_awq_forward(h, X, M: int, Y, stream=None) -> None:
    _check(lib().svdq_awq_forward(h, _ptr(X), M, _ptr(Y), _stream(stream)), "svdq_awq_forward")


class AwqLinear:
    """One awq_w4a16 layer (4-bit weights, bf16 activations) on `device` (default:
    the current CUDA device), built from canonical prepared weights
    (svdq_awq_prepare output or a dict with the same arrays); `forward(x)` maps
    bf16 [M, K] to bf16 [M, N], enqueued with the layer's device current."""

    def __init__(self, canonical: dict, device=None):
        import torch

        self.N, self.K = int(canonical["N"]), int(canonical["K"])
        self.device = _layer_device(device)
        self.blob = torch.from_numpy(svdq_awq_pack(canonical)).to(self.device)
        with torch.cuda.device(self.device):
            self.handle = svdq_awq_layer_create(self.blob, self.blob.numel(), self.N, self.K)

    def forward(self, x, out=None, stream=None):
        import torch

        _check_input(x, self.K, self.device)
        M = x.numel() // self.K
        with torch.cuda.device(self.device), _on(stream if out is None else None, self.device):
            y = out if out is not None else torch.empty(M, self.N, dtype=torch.bfloat16, device=x.device)
            svdq_awq_forward(self.handle, x, M, y, stream)
        return y

    __call__ = forward

    def status(self) -> int:
        return svdq_awq_read_status(self.handle)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.svdq_awq_layer_destroy(h)
            self.handle = None


# ----------------------------------------------------------------------------- int8 tensorwise W8A8
def svdq_w8a8_prepare(W):
    """Host: W [N,K] bf16 bits -> (int8 codes [N,K], s_w)."""
    W = np.ascontiguousarray(W, np.uint16)
    N, K = W.shape
    codes = np.empty((N, K), np.int8)
    s = ctypes.c_float()
    _check(lib().svdq_w8a8_prepare(W.ctypes.data, N, K, codes.ctypes.data, ctypes.byref(s)), "svdq_w8a8_prepare")
    return codes, float(s.value)


def svdq_w8a8_packed_size(N: int, K: int) -> int:
    v = ctypes.c_size_t()
    _check(lib().svdq_w8a8_packed_size(N, K, ctypes.byref(v)), "svdq_w8a8_packed_size")
    return v.value


def svdq_w8a8_pack(wcodes, bias=None) -> np.ndarray:
    wcodes = np.ascontiguousarray(wcodes, np.int8)
    N, K = wcodes.shape
    size = svdq_w8a8_packed_size(N, K)
    blob = np.zeros(size, np.uint8)
    b = None if bias is None else np.ascontiguousarray(bias, np.uint16)
    _check(lib().svdq_w8a8_pack(N, K, wcodes.ctypes.data, None if b is None else b.ctypes.data, blob.ctypes.data,
                                size), "svdq_w8a8_pack")
    return blob


def svdq_w8a8_layer_create(dev_blob, blob_bytes: int, N: int, K: int, s_w: float):
    h = ctypes.c_void_p()
    _check(lib().svdq_w8a8_layer_create(_ptr(dev_blob), blob_bytes, N, K, s_w, ctypes.byref(h)),
           "svdq_w8a8_layer_create")
    return h


def svdq_w8a8_layer_destroy(h) -> None:
    lib().svdq_w8a8_layer_destroy(h)


def svdq_w8a8_workspace_size(h, M: int) -> int:
    v = ctypes.c_size_t()
    _check(lib().svdq_w8a8_workspace_size(h, M, ctypes.byref(v)), "svdq_w8a8_workspace_size")
    return v.value


def svdq_w8a8_quantize_act(h, X, M: int, ws, stream=None) -> None:
    _check(lib().svdq_w8a8_quantize_act(h, _ptr(X), M, _ptr(ws), ws.numel(), _stream(stream)),
           "svdq_w8a8_quantize_act")


def svdq_w8a8_gemm(h, M: int, Y, ws, stream=None) -> None:
    _check(lib().svdq_w8a8_gemm(h, M, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)), "svdq_w8a8_gemm")


def svdq_w8a8_forward(h, X, M: int, Y, ws, stream=None) -> None:
    _check(lib().svdq_w8a8_forward(h, _ptr(X), M, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)),
           "svdq_w8a8_forward")


def svdq_w8a8_read_status(h, M: int, ws) -> int:
    v = ctypes.c_int()
    _check(lib().svdq_w8a8_read_status(h, M, _ptr(ws), ws.numel(), ctypes.byref(v)), "svdq_w8a8_read_status")
    return v.value


class W8A8Linear:
    """One INT8 tensorwise W8A8 layer on `device` (default: the current CUDA
    device), from prepared int8 weight codes [N,K], the weight scale s_w and an
    optional bf16 bias; `forward(x)` maps bf16 [M, K] to bf16 [M, N], enqueued
    with the layer's device current."""

    def __init__(self, wcodes, s_w: float, bias=None, device=None):
        import torch

        self.N, self.K = int(wcodes.shape[0]), int(wcodes.shape[1])
        self.s_w = float(s_w)
        self.device = _layer_device(device)
        self.blob = torch.from_numpy(svdq_w8a8_pack(wcodes, bias)).to(self.device)
        with torch.cuda.device(self.device):
            self.handle = svdq_w8a8_layer_create(self.blob, self.blob.numel(), self.N, self.K, self.s_w)
        self._ws = {}

    def workspace_size(self, M: int) -> int:
        return svdq_w8a8_workspace_size(self.handle, M)

    def workspace(self, M: int):
        import torch

        if M not in self._ws:
            self._ws[M] = torch.empty(self.workspace_size(M), dtype=torch.uint8, device=self.device)
        return self._ws[M]

    def quantize_act(self, x, M: int, stream=None):
        import torch

        with torch.cuda.device(self.device), _on(stream if M not in self._ws else None, self.device):
            svdq_w8a8_quantize_act(self.handle, x, M, self.workspace(M), stream)

    def gemm(self, M: int, y, stream=None):
        import torch

        with torch.cuda.device(self.device), _on(stream if M not in self._ws else None, self.device):
            svdq_w8a8_gemm(self.handle, M, y, self.workspace(M), stream)

    def forward(self, x, out=None, stream=None):
        import torch

        _check_input(x, self.K, self.device)
        M = x.numel() // self.K
        with torch.cuda.device(self.device), _on(stream if out is None or M not in self._ws else None, self.device):
            y = out if out is not None else torch.empty(M, self.N, dtype=torch.bfloat16, device=x.device)
            svdq_w8a8_forward(self.handle, x, M, y, self.workspace(M), stream)
        return y

    __call__ = forward

    def status(self, M: int) -> int:
        return svdq_w8a8_read_status(self.handle, M, self.workspace(M))

    def read_act(self, M: int):
        """Activation codes int8 [M, K] and s_x from the workspace (after quantize_act)."""
        ws = self.workspace(M).cpu().numpy()
        ctrl = (M * self.K + 1023) // 1024 * 1024
        return dict(codes=ws[:M * self.K].view(np.int8).reshape(M, self.K).copy(),
                    s_x=np.float32(ws[ctrl + 4:ctrl + 8].view(np.float32)[0]))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.svdq_w8a8_layer_destroy(h)
            self.handle = None


# ----------------------------------------------------------------------------- FP8, one scale for each block of 128
def svdq_fp8_prepare(W):
    """Host: W [N,K] bf16 bits -> (E4M3 codes u8 [N,K], scales f32 [ceil(N/128), ceil(K/128)])."""
    W = np.ascontiguousarray(W, np.uint16)
    N, K = W.shape
    codes = np.empty((N, K), np.uint8)
    scales = np.empty(((N + 127) // 128, (K + 127) // 128), np.float32)
    _check(lib().svdq_fp8_prepare(W.ctypes.data, N, K, codes.ctypes.data, scales.ctypes.data), "svdq_fp8_prepare")
    return codes, scales


def svdq_fp8_packed_size(N: int, K: int) -> int:
    v = ctypes.c_size_t()
    _check(lib().svdq_fp8_packed_size(N, K, ctypes.byref(v)), "svdq_fp8_packed_size")
    return v.value


def svdq_fp8_pack(wcodes, wscales, bias=None) -> np.ndarray:
    wcodes = np.ascontiguousarray(wcodes, np.uint8)
    wscales = np.ascontiguousarray(wscales, np.float32)
    N, K = wcodes.shape
    if wscales.shape != ((N + 127) // 128, (K + 127) // 128):
        raise ValueError(f"expected scales [{(N + 127) // 128}, {(K + 127) // 128}], got {wscales.shape}")
    b = None if bias is None else np.ascontiguousarray(bias, np.uint16)
    if b is not None and b.shape != (N,):
        raise ValueError(f"expected a bias [{N}], got {b.shape}")
    size = svdq_fp8_packed_size(N, K)
    blob = np.empty(size, np.uint8)
    _check(lib().svdq_fp8_pack(N, K, wcodes.ctypes.data, wscales.ctypes.data, None if b is None else b.ctypes.data,
                               blob.ctypes.data, size), "svdq_fp8_pack")
    return blob


def svdq_fp8_layer_create(dev_blob, blob_bytes: int, N: int, K: int):
    h = ctypes.c_void_p()
    _check(lib().svdq_fp8_layer_create(_ptr(dev_blob), blob_bytes, N, K, ctypes.byref(h)), "svdq_fp8_layer_create")
    return h


def svdq_fp8_layer_destroy(h) -> None:
    lib().svdq_fp8_layer_destroy(h)


def svdq_fp8_workspace_size(h, M: int) -> int:
    v = ctypes.c_size_t()
    _check(lib().svdq_fp8_workspace_size(h, M, ctypes.byref(v)), "svdq_fp8_workspace_size")
    return v.value


def svdq_fp8_quantize_act(h, X, M: int, ws, stream=None) -> None:
    _check(lib().svdq_fp8_quantize_act(h, _ptr(X), M, _ptr(ws), ws.numel(), _stream(stream)), "svdq_fp8_quantize_act")


def svdq_fp8_gemm(h, M: int, Y, ws, stream=None) -> None:
    _check(lib().svdq_fp8_gemm(h, M, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)), "svdq_fp8_gemm")


def svdq_fp8_forward(h, X, M: int, Y, ws, stream=None) -> None:
    st = lib().svdq_fp8_forward(h, _ptr(X), M, _ptr(Y), ws.data_ptr(), ws.numel(), _stream(stream))
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_fp8_forward")


def svdq_fp8_read_status(h, M: int, ws) -> int:
    v = ctypes.c_int()
    _check(lib().svdq_fp8_read_status(h, M, _ptr(ws), ws.numel(), ctypes.byref(v)), "svdq_fp8_read_status")
    return v.value


class Fp8Linear:
    """One FP8 layer with a scale for each block of 128, on `device` (default: the
    current CUDA device), from E4M3 weight codes u8 [N,K] (svdq_fp8_prepare, or a
    checkpoint's own), their scales f32 [ceil(N/128), ceil(K/128)] and an optional
    bf16 bias (bits); `forward(x)` maps bf16 [M, K] to bf16 [M, N], enqueued with the
    layer's device current.  One workspace serves every token count, and one call at
    a time (calls on several streams take one layer object each): a call with more
    tokens than any before makes a larger one, memory of the stream it runs on, and
    the smaller stay, as a captured graph may use them."""

    def __init__(self, wcodes, wscales, bias=None, device=None):
        import torch

        self.N, self.K = int(wcodes.shape[0]), int(wcodes.shape[1])
        self.device = _layer_device(device)
        self.blob = torch.from_numpy(svdq_fp8_pack(wcodes, wscales, bias)).to(self.device)
        with torch.cuda.device(self.device):
            self.handle = svdq_fp8_layer_create(self.blob, self.blob.numel(), self.N, self.K)
        self._handle = self.handle.value
        self._blob_stream = torch.cuda.current_stream(self.device).cuda_stream
        self._room = None  # (buffer, handle of the stream whose memory it is, weights, theirs)
        self._smaller = []

    def workspace_size(self, M: int) -> int:
        return svdq_fp8_workspace_size(self.handle, M)

    def workspace(self, M: int):
        """The workspace of a call with M tokens: the end of the buffer, so that the status word, a workspace's last 16
        bytes, has one place whatever M."""
        size = self.workspace_size(M)
        have = self._room[0].numel() if self._room else 0
        if have < size:
            torch = _torch()
            # Half as much again as the one before: all of them come to 4.5 times what the largest call needs at most.
            buf = torch.empty(16 + max(size - 16, (have // 1024 * 3 + 1) // 2 * 1024), dtype=torch.uint8, device=self.device)
            buf[-16:].zero_()  # no call yet: status 0
            if self._room:
                self._smaller.append(self._room)
            self._room = buf, torch.cuda.current_stream(self.device).cuda_stream, self.blob, self._blob_stream
        buf = self._room[0]
        return buf[buf.numel() - size:]

    def forward(self, x, out=None, stream=None):
        forward = (_calls_module or _calls()).fp8_forward
        if stream is not None:
            if out is not None and isinstance(stream, _torch().cuda.Stream) and stream.device == self.device:
                y = forward(self._handle, self.N, self.K, self.device.index, self._room, x, out, stream.cuda_stream,
                            stream.stream_id)
                if y is not None:
                    return y
            with _stream_context(stream, self.device):  # what the call allocates is memory of the stream that writes it
                return self.forward(x, out)
        y = forward(self._handle, self.N, self.K, self.device.index, self._room, x, out, None, None)
        if y is None:  # the first call with so many tokens
            self.workspace(x.numel() // self.K)
            y = forward(self._handle, self.N, self.K, self.device.index, self._room, x, out, None, None)
        return y

    __call__ = forward

    def status(self, M: int) -> int:
        """The status word of the layer's last call, which has to be done."""
        return svdq_fp8_read_status(self.handle, M, self.workspace(M))

    def read_act(self, M: int):
        """Activation codes u8 [M, K] and scales f32 [M, ceil(K/128)] of the layer's last call, which had M tokens."""
        ws = self.workspace(M).cpu().numpy()
        kb = (self.K + 127) // 128
        ld = (kb + 3) // 4 * 4
        at = (M * self.K + 1023) // 1024 * 1024
        scales = ws[at:at + 4 * M * ld].view(np.float32).reshape(M, ld)[:, :kb]
        return dict(codes=ws[:M * self.K].reshape(M, self.K).copy(), scales=scales.copy())

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.svdq_fp8_layer_destroy(h)
            self.handle = None


# ----------------------------------------------------------------------------- between the projections
PAIRS = {"interleaved": 0, "halves": 1}
_attn_status = {}


_calls_module = None


def _calls():
    """The module _marshal.so (tensors to the library's arguments), bound to the loaded library; raises if it was not
    built (no fallback)."""
    global _calls_module
    if _calls_module is None:
        torch, L = _torch(), lib()
        try:
            from . import _marshal as m
        except ImportError as e:
            raise RuntimeError(f"_marshal.so is missing or does not load ({e}): build it with "
                               "`python -m diffusion_transformer_w4a4_b200.build`") from e
        address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
        m.bind(address(L.svdq_qk_norm_rope), address(L.svdq_cross_attn), address(L.svdq_fp8_forward),
               address(L.svdq_fp8_workspace_size), SvdqError, attn_status, torch.OutOfMemoryError,
               str(torch.__version__))
        _calls_module = m
    return _calls_module


def attn_status(device=None):
    """The status word (int32 tensor of one element) that svdq_cross_attn and svdq_qk_norm_rope report to on
    `device`, unless they are given another: 0, or the code of the first device-side failure (sticky)."""
    torch = _torch()
    device = _layer_device(device)
    t = _attn_status.get(device.index)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first call on a device makes its status word: make it before any stream capture")
        with torch.cuda.device(device):
            t = torch.zeros(1, dtype=torch.int32, device=device)
            torch.cuda.current_stream().synchronize()  # before any other stream uses it
        _attn_status[device.index] = t
        _calls().set_status(device.index, t.data_ptr())
    return t


def svdq_qk_norm_rope(q, k=None, q_weight=None, k_weight=None, *, eps=1e-6, rope=None, positions=None,
                      pairs="interleaved", out_q=None, out_k=None, status=None, stream=None):
    """RMS norm of each head of q [B,S,H,D] (and k, in the same launch) with an optional weight bf16 [D], then the
    rotation by `rope` f32 [rows, rot/2, 2] (cosine, sine; the first rot elements of a head, in `pairs`
    "interleaved" or "halves"): row positions[b, s] (int32 [B,S]), or row s without positions.  Any strided view
    with contiguous heads (a slice of a fused projection's output); out_q / out_k may be q / k themselves.  Returns
    the rotated q, or (q, k)."""
    if stream is not None:
        out_q = _empty_like(q, stream) if out_q is None else out_q
        out_k = _empty_like(k, stream) if out_k is None and k is not None else out_k
        stream = _stream(stream)
    return (_calls_module or _calls()).qk_norm_rope(q, k, q_weight, k_weight, eps, rope, positions, PAIRS[pairs],
                                                        out_q, out_k, status, stream)


def svdq_cross_attn(q, k, v, *, kv_len=None, kv_mask=None, scale=None, out=None, status=None, stream=None):
    """Attention of q [B,Sq,H,D] over k, v [B,Sk,Hkv,D] (bf16 views, contiguous heads; H a multiple of Hkv; batch
    and heads of k and v may be expanded): softmax(scale q k^T) v over the first kv_len[b] keys (int32 [B]) with
    kv_mask[b, t] nonzero (uint8 or bool [B,Sk]).  Rows without a key give 0.  scale defaults to 1/sqrt(D).
    Returns bf16 [B,Sq,H,D]."""
    if stream is not None:
        out = _empty_like(q, stream) if out is None else out
        stream = _stream(stream)
    return (_calls_module or _calls()).cross_attn(q, k, v, kv_len, kv_mask, scale, out, status, stream)
