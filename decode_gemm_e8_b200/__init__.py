"""E8 lattice-codebook weights decoded on a B200 and fed into a bf16 GEMM.

Thin ctypes binding over ``libe8.so`` (C ABI in ``include/e8.h``).  The
functions carry the C names and only marshal arguments: tensors become device
pointers, the current torch CUDA stream becomes the ``stream`` argument, and
nonzero status codes raise :class:`E8Error`.  Every step of the computation
runs in the library's CUDA kernels; if the library is missing this module
raises instead of computing anything another way.

Method: page "glq 0.1.1" on PyPI, "How it works" (E8 codebook of 65536 vectors
from the first 7 shells, 16-bit index per 8 weights plus an 8/16-bit residual
index at 3/4 bpw, randomized Hadamard transform, Euclidean nearest codebook
vector) and the "Bit widths" table (one global scale per layer).
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libe8.so")

E8_OK, E8_EINVAL, E8_EWORKSPACE, E8_EDEVICE, E8_ECUDA, E8_ETIMEOUT, E8_ENOMEM, E8_EDATA = range(8)
E8_EP_BLOCK_GROUPS = 64
E8_EP_TABLE_WORDS = 770
E8_GEMM_AUTO, E8_GEMM_ACT_RHT, E8_GEMM_DECODED_W, E8_GEMM_ACT_RHT_SMEM, E8_GEMM_SIMT = range(5)
E8_OP_ENCODE = 100
E8_DT_BF16, E8_DT_F16, E8_DT_F32 = range(3)
E8_MOE_MAX_TOKENS, E8_MOE_MAX_EXPERTS, E8_MOE_MAX_TOPK = 64, 512, 16

# every symbol include/e8.h declares
EXPORTED = ("e8_codebook_build", "e8_codebook_free", "e8_codebook_export", "e8_rht_forward",
            "e8_encode", "e8_decode_to_bf16", "e8_act_rht", "e8_act_rht_q8", "e8_act_q8_bytes",
            "e8_gemm", "e8_gemm_xt",
            "e8_gemm_xt_rows", "e8_gemm_act_noalloc", "e8_gemm_host",
            "e8_gemm_grouped", "e8_gemm_grouped_workspace_bytes",
            "e8_rht_forward_nh", "e8_encode_nh", "e8_decode_to_bf16_nh", "e8_gemm_nh",
            "e8_workspace_bytes_nh",
            "e8_gemm_host_workspace_bytes", "e8_gemm_auto_mode",
            "e8_workspace_bytes", "e8_sync_status", "e8_debug_wait_timeout", "e8_status_str",
            "e8_version",
            "e8_ep_num_blocks", "e8_ep_max_words", "e8_ep_actual_bpp",
            "e8_ep_encode_workspace_bytes", "e8_ep_gemm_workspace_bytes", "e8_ep_encode",
            "e8_ep_estimate_bpp", "e8_ep_choose_delta", "e8_ep_decode_to_bf16", "e8_ep_gemm",
            "e8_mx4_code_bytes", "e8_mx4_scale_bytes", "e8_mx4_encode", "e8_mx4_decode_to_bf16",
            "e8_mx4_gemm_codes", "e8_mx4_gemm", "e8_mx4_gemm_codes_workspace_bytes",
            "e8_mx4_gemm_workspace_bytes", "e8_mx4_moe", "e8_mx4_moe_workspace_bytes")

_lib = None


class E8Error(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (where, status_str(code), code))


def load_library(path: str = LIB_PATH):
    """Loads libe8.so and declares argument types.  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libe8.so not built (%s); run `python -m decode_gemm_e8_b200.build`" % path)
    lib = ctypes.CDLL(path)
    c = ctypes
    P, I64, U64 = c.c_void_p, c.c_int64, c.c_uint64
    sig = {
        "e8_codebook_build": ([c.POINTER(c.c_void_p), c.c_int], c.c_int),
        "e8_codebook_free": ([P], None),
        "e8_codebook_export": ([P, P], c.c_int),
        "e8_rht_forward": ([P, P, I64, I64, U64, c.c_float, P, P], c.c_int),
        "e8_encode": ([P, P, I64, I64, c.c_int, U64, c.c_float, P, P, P, c.c_size_t, P], c.c_int),
        "e8_decode_to_bf16": ([P, P, P, I64, I64, c.c_int, U64, c.c_float, P, P], c.c_int),
        "e8_act_rht": ([P, I64, I64, U64, P, I64, P], c.c_int),
        "e8_gemm": ([P, P, I64, P, P, I64, I64, c.c_int, U64, c.c_float, P, c.c_int, P,
                     c.c_size_t, P], c.c_int),
        "e8_act_rht_q8": ([P, I64, I64, U64, P, P], c.c_int),
        "e8_act_q8_bytes": ([I64, I64], c.c_size_t),
        "e8_gemm_xt": ([P, P, I64, P, P, I64, I64, c.c_int, c.c_float, P, P], c.c_int),
        "e8_gemm_xt_rows": ([I64], c.c_int),
        "e8_gemm_act_noalloc": ([P, P, I64, P, P, I64, I64, c.c_int, U64, c.c_float, P, P],
                                c.c_int),
        "e8_gemm_host": ([P, P, I64, P, P, I64, I64, c.c_int, U64, c.c_float, P, c.c_int, P,
                          c.c_size_t, P], c.c_int),
        "e8_gemm_host_workspace_bytes": ([c.c_int, I64, I64, I64, c.c_int], c.c_size_t),
        "e8_gemm_auto_mode": ([I64, I64, I64, c.c_int], c.c_int),
        "e8_gemm_grouped": ([P, P, I64, I64, c.c_int, P, c.c_int, P, c.c_size_t, P], c.c_int),
        "e8_rht_forward_nh": ([P, P, I64, I64, I64, U64, c.c_float, P, P], c.c_int),
        "e8_encode_nh": ([P, P, I64, I64, I64, c.c_int, U64, c.c_float, P, P, P, c.c_size_t, P],
                         c.c_int),
        "e8_decode_to_bf16_nh": ([P, P, P, I64, I64, I64, c.c_int, U64, c.c_float, P, P],
                                 c.c_int),
        "e8_gemm_nh": ([P, P, I64, P, P, I64, I64, I64, c.c_int, U64, c.c_float, P, c.c_int, P,
                        c.c_size_t, P], c.c_int),
        "e8_workspace_bytes_nh": ([c.c_int, I64, I64, I64, I64, c.c_int], c.c_size_t),
        "e8_gemm_grouped_workspace_bytes": ([I64, I64, c.c_int, c.c_int], c.c_size_t),
        "e8_workspace_bytes": ([c.c_int, I64, I64, I64, c.c_int], c.c_size_t),
        "e8_sync_status": ([P, P], c.c_int),
        "e8_debug_wait_timeout": ([P, c.c_int, P], c.c_int),
        "e8_status_str": ([c.c_int], c.c_char_p),
        "e8_version": ([], c.c_int),
        "e8_ep_num_blocks": ([I64, I64], I64),
        "e8_ep_max_words": ([I64, I64], I64),
        "e8_ep_actual_bpp": ([I64, I64, I64], c.c_double),
        "e8_ep_encode_workspace_bytes": ([I64, I64], c.c_size_t),
        "e8_ep_gemm_workspace_bytes": ([I64, I64, I64], c.c_size_t),
        "e8_ep_encode": ([P, P, I64, I64, c.c_float, P, I64, P, P, P, c.POINTER(c.c_int64), P,
                          c.c_size_t, P], c.c_int),
        "e8_ep_estimate_bpp": ([P, P, I64, I64, c.c_float, c.POINTER(c.c_double), P, c.c_size_t,
                                P], c.c_int),
        "e8_ep_choose_delta": ([P, P, I64, I64, c.c_double, c.POINTER(c.c_float), P, c.c_size_t,
                                P], c.c_int),
        "e8_ep_decode_to_bf16": ([P, P, I64, P, P, P, I64, I64, P, P], c.c_int),
        "e8_ep_gemm": ([P, P, I64, P, I64, P, P, P, I64, I64, P, P, c.c_size_t, P], c.c_int),
        "e8_mx4_code_bytes": ([I64, I64], I64),
        "e8_mx4_scale_bytes": ([I64, I64], I64),
        "e8_mx4_encode": ([P, P, c.c_int, I64, I64, I64, I64, P, P, P], c.c_int),
        "e8_mx4_decode_to_bf16": ([P, P, P, I64, I64, I64, P, P], c.c_int),
        "e8_mx4_gemm_codes": ([P, P, P, I64, P, P, I64, I64, P, P, c.c_size_t, P], c.c_int),
        "e8_mx4_gemm_codes_workspace_bytes": ([I64, I64, I64], c.c_size_t),
        "e8_mx4_gemm": ([P, P, c.c_int, I64, I64, P, P, I64, I64, P, P, c.c_size_t, P], c.c_int),
        "e8_mx4_gemm_workspace_bytes": ([I64, I64, I64], c.c_size_t),
        "e8_mx4_moe": ([P, P, I64, I64, P, I64, c.c_int, c.c_int, P, P, I64, P, P, P, P, P, P,
                        c.c_size_t, P], c.c_int),
        "e8_mx4_moe_workspace_bytes": ([I64, I64, I64, c.c_int, I64], c.c_size_t),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


E8_GROUP_MAX = 4


class GemmItem(ctypes.Structure):
    """struct e8_gemm_item of include/e8.h."""
    _fields_ = [("idx1", ctypes.c_void_p), ("idx2", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("rht_seed", ctypes.c_uint64), ("scale", ctypes.c_float),
                ("Y", ctypes.c_void_p)]


def status_str(code: int) -> str:
    return load_library().e8_status_str(int(code)).decode()


def _check(rc: int, where: str):
    if rc != E8_OK:
        raise E8Error(rc, where)


def _ptr(t):
    # the argtypes declare c_void_p, which takes a plain integer address
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    if stream is not None:
        return stream.cuda_stream
    try:
        # the raw handle of the current stream, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


class Codebook:
    """Device-resident canonical codebook tables (``e8_codebook_build``)."""

    def __init__(self, device: int = 0):
        lib = load_library()
        h = ctypes.c_void_p()
        _check(lib.e8_codebook_build(ctypes.byref(h), int(device)), "e8_codebook_build")
        self._h = h
        self.device = int(device)

    @property
    def handle(self):
        return self._h

    def free(self):
        if getattr(self, "_h", None):
            load_library().e8_codebook_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def e8_codebook_build(device: int = 0) -> Codebook:
    return Codebook(device)


def e8_codebook_free(cb: Codebook) -> None:
    cb.free()


def e8_codebook_export(cb: Codebook):
    """The 65536 codebook vectors as an int8 numpy array [65536, 8] of doubled coordinates."""
    import numpy as np
    out = np.zeros((65536, 8), dtype=np.int8)
    _check(load_library().e8_codebook_export(cb.handle, ctypes.c_void_p(out.ctypes.data)),
           "e8_codebook_export")
    return out


def e8_rht_forward(cb: Codebook, W, rht_seed: int, scale: float, U=None, stream=None, nh=None):
    """nh: explicit Hadamard block (e8_rht_forward_nh); None for the default."""
    import torch
    N, K = W.shape
    if U is None:
        U = torch.empty_like(W)
    lib = load_library()
    if nh is None:
        rc = lib.e8_rht_forward(cb.handle, _ptr(W), N, K, int(rht_seed) & (2**64 - 1),
                                float(scale), _ptr(U), _stream(stream))
    else:
        rc = lib.e8_rht_forward_nh(cb.handle, _ptr(W), N, K, int(nh), int(rht_seed) & (2**64 - 1),
                                   float(scale), _ptr(U), _stream(stream))
    _check(rc, "e8_rht_forward")
    return U


def e8_workspace_bytes(op: int, M: int, N: int, K: int, bpw: int, nh=None) -> int:
    if nh is not None:
        return int(load_library().e8_workspace_bytes_nh(int(op), int(M), int(N), int(K), int(nh),
                                                        int(bpw)))
    return int(load_library().e8_workspace_bytes(int(op), int(M), int(N), int(K), int(bpw)))


def e8_gemm_auto_mode(M: int, N: int, K: int, bpw: int) -> int:
    return int(load_library().e8_gemm_auto_mode(int(M), int(N), int(K), int(bpw)))


def _workspace(nbytes: int, device, workspace=None):
    import torch
    if workspace is not None:
        return workspace
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def e8_encode(cb: Codebook, W, bpw: int, rht_seed: int, scale: float, idx1=None, idx2=None,
              workspace=None, stream=None, nh=None):
    """W fp32 [N, K] (CUDA) -> (idx1 uint16 [N, K/8], idx2 uint8/uint16 [N, K/8] or None).
    nh: explicit Hadamard block (e8_encode_nh); None for the default."""
    import torch
    N, K = W.shape
    dev = W.device
    if idx1 is None:
        idx1 = torch.empty((N, K // 8), dtype=torch.uint16, device=dev)
    if idx2 is None and bpw > 2:
        idx2 = torch.empty((N, K // 8), dtype=torch.uint8 if bpw == 3 else torch.uint16, device=dev)
    need = e8_workspace_bytes(E8_OP_ENCODE, 0, N, K, bpw)
    ws = _workspace(need, dev, workspace)
    lib = load_library()
    if nh is None:
        rc = lib.e8_encode(cb.handle, _ptr(W), N, K, int(bpw), int(rht_seed) & (2**64 - 1),
                           float(scale), _ptr(idx1), _ptr(idx2), _ptr(ws), ws.numel(),
                           _stream(stream))
    else:
        rc = lib.e8_encode_nh(cb.handle, _ptr(W), N, K, int(nh), int(bpw),
                              int(rht_seed) & (2**64 - 1), float(scale), _ptr(idx1), _ptr(idx2),
                              _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "e8_encode")
    return idx1, idx2


def e8_decode_to_bf16(cb: Codebook, idx1, idx2, N: int, K: int, bpw: int, rht_seed: int,
                      scale: float, out=None, stream=None, nh=None):
    """Decoded weights, torch.bfloat16 [N, K] on the device of idx1.
    nh: explicit Hadamard block (e8_decode_to_bf16_nh); None for the default."""
    import torch
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=idx1.device)
    lib = load_library()
    if nh is None:
        rc = lib.e8_decode_to_bf16(cb.handle, _ptr(idx1), _ptr(idx2), N, K, int(bpw),
                                   int(rht_seed) & (2**64 - 1), float(scale), _ptr(out),
                                   _stream(stream))
    else:
        rc = lib.e8_decode_to_bf16_nh(cb.handle, _ptr(idx1), _ptr(idx2), N, K, int(nh), int(bpw),
                                      int(rht_seed) & (2**64 - 1), float(scale), _ptr(out),
                                      _stream(stream))
    _check(rc, "e8_decode_to_bf16")
    return out


def e8_act_rht(X, rht_seed: int, rows: int | None = None, out=None, stream=None):
    """X bf16 [M, K] -> Xt bf16 [rows, K] (hi rows, lo rows, zero padding)."""
    import torch
    M, K = X.shape
    rows = 2 * M if rows is None else int(rows)
    if out is None:
        out = torch.empty((rows, K), dtype=torch.bfloat16, device=X.device)
    _check(load_library().e8_act_rht(_ptr(X), M, K, int(rht_seed) & (2**64 - 1), _ptr(out), rows,
                                     _stream(stream)), "e8_act_rht")
    return out


def e8_gemm(cb: Codebook, X, idx1, idx2, N: int, K: int, bpw: int, rht_seed: int, scale: float,
            mode: int = E8_GEMM_AUTO, Y=None, workspace=None, stream=None, nh=None):
    """Y fp32 [M, N] = X bf16 [M, K] times the decoded weights transposed.
    nh: explicit Hadamard block (e8_gemm_nh); None for the default."""
    import torch
    M = X.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=dev)
    # a caller's workspace is checked by the library (E8_EWORKSPACE if too small)
    ws = workspace if workspace is not None else _workspace(
        e8_workspace_bytes(mode, M, N, K, bpw, nh), dev)
    lib = load_library()
    if nh is None:
        rc = lib.e8_gemm(cb.handle, _ptr(X), M, _ptr(idx1), _ptr(idx2), N, K, int(bpw),
                         int(rht_seed) & (2**64 - 1), float(scale), _ptr(Y), int(mode),
                         _ptr(ws), ws.numel(), _stream(stream))
    else:
        rc = lib.e8_gemm_nh(cb.handle, _ptr(X), M, _ptr(idx1), _ptr(idx2), N, K, int(nh),
                            int(bpw), int(rht_seed) & (2**64 - 1), float(scale), _ptr(Y),
                            int(mode), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "e8_gemm")
    return Y


def e8_gemm_host_workspace_bytes(mode: int, M: int, N: int, K: int, bpw: int) -> int:
    return int(load_library().e8_gemm_host_workspace_bytes(int(mode), int(M), int(N), int(K),
                                                           int(bpw)))


def _host_ptr(a):
    # torch CPU tensor or numpy array
    return a.data_ptr() if hasattr(a, "data_ptr") else a.ctypes.data


def e8_gemm_host(cb: Codebook, X_host, idx1, idx2, N: int, K: int, bpw: int, rht_seed: int,
                 scale: float, Y_host=None, mode: int = E8_GEMM_AUTO, workspace=None,
                 stream=None):
    """e8_gemm with X (bf16 [M, K]) and Y (fp32 [M, N]) in host memory.

    One library call queues the copy of X in, the product and the copy of Y
    out on the stream; Y_host holds the product once the stream has passed it.
    X_host: a torch bf16/int16 CPU tensor or a numpy uint16/int16 array.
    A new page-locked Y_host is made when None is given."""
    import torch
    M = X_host.shape[0]
    if Y_host is None:
        Y_host = torch.empty((M, N), dtype=torch.float32).pin_memory()
    ws = workspace if workspace is not None else _workspace(
        e8_gemm_host_workspace_bytes(mode, M, N, K, bpw), torch.device("cuda", cb.device))
    _check(load_library().e8_gemm_host(cb.handle, _host_ptr(X_host), M, _ptr(idx1), _ptr(idx2),
                                       N, K, int(bpw), int(rht_seed) & (2**64 - 1), float(scale),
                                       _host_ptr(Y_host), int(mode), _ptr(ws), ws.numel(),
                                       _stream(stream)), "e8_gemm_host")
    return Y_host


def e8_gemm_xt_rows(M: int) -> int:
    return int(load_library().e8_gemm_xt_rows(int(M)))


def e8_act_q8_bytes(M: int, K: int) -> int:
    return int(load_library().e8_act_q8_bytes(int(M), int(K)))


def e8_act_rht_q8(X, rht_seed: int, out=None, stream=None):
    """X bf16 [M, K] -> the int8 activation buffer (uint8 tensor) of e8_gemm_xt."""
    import torch
    M, K = X.shape
    if out is None:
        out = torch.empty(max(16, e8_act_q8_bytes(M, K)), dtype=torch.uint8, device=X.device)
    _check(load_library().e8_act_rht_q8(_ptr(X), M, K, int(rht_seed) & (2**64 - 1), _ptr(out),
                                        _stream(stream)), "e8_act_rht_q8")
    return out


def e8_gemm_xt(cb: Codebook, xq, M: int, idx1, idx2, N: int, K: int, bpw: int, scale: float,
               Y=None, stream=None):
    """Fused decode + int8 GEMM on a buffer from e8_act_rht_q8; the product is
    added into Y (a new zero tensor when Y is None)."""
    import torch
    if Y is None:
        Y = torch.zeros((M, N), dtype=torch.float32, device=xq.device)
    _check(load_library().e8_gemm_xt(cb.handle, _ptr(xq), int(M), _ptr(idx1), _ptr(idx2), int(N),
                                     int(K), int(bpw), float(scale), _ptr(Y), _stream(stream)),
           "e8_gemm_xt")
    return Y


def e8_gemm_act_noalloc(cb: Codebook, X, idx1, idx2, N: int, K: int, bpw: int, rht_seed: int,
                        scale: float, Y, stream=None):
    """E8_GEMM_ACT_RHT with the library's fixed scratch array instead of a workspace.

    For callers that may not allocate device memory when they run the layer (CUDA
    graph capture, framework-owned memory, latency-critical loops).  Y must be
    given: this call allocates nothing."""
    _check(load_library().e8_gemm_act_noalloc(cb.handle, _ptr(X), X.shape[0], _ptr(idx1),
                                              _ptr(idx2), int(N), int(K), int(bpw),
                                              int(rht_seed) & (2**64 - 1), float(scale), _ptr(Y),
                                              _stream(stream)), "e8_gemm_act_noalloc")
    return Y


def e8_sync_status(cb: Codebook, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status as a status code."""
    return int(load_library().e8_sync_status(cb.handle, _stream(stream)))


def e8_debug_wait_timeout(cb: Codebook, wait_ms: int, stream=None) -> None:
    _check(load_library().e8_debug_wait_timeout(cb.handle, int(wait_ms), _stream(stream)),
           "e8_debug_wait_timeout")


def e8_version() -> int:
    return int(load_library().e8_version())


def e8_gemm_grouped_workspace_bytes(M: int, K: int, bpw: int, count: int) -> int:
    return int(load_library().e8_gemm_grouped_workspace_bytes(int(M), int(K), int(bpw),
                                                              int(count)))


def e8_gemm_grouped(cb: Codebook, X, items, K: int, bpw: int, workspace=None, stream=None):
    """Y_i = X W_dec_i^T for several weight matrices that read the same X.

    items: sequence of (idx1, idx2, N, rht_seed, scale) or
    (idx1, idx2, N, rht_seed, scale, Y); a missing Y is allocated (fp32 [M, N]).
    Returns the list of Y tensors."""
    import torch
    M = int(X.shape[0])
    arr = (GemmItem * max(1, len(items)))()
    outs = []
    for i, it in enumerate(items):
        idx1, idx2, N, rs, scale = it[:5]
        Y = it[5] if len(it) > 5 and it[5] is not None else torch.empty(
            (M, int(N)), dtype=torch.float32, device=X.device)
        outs.append(Y)
        arr[i] = GemmItem(_ptr(idx1), _ptr(idx2), int(N), int(rs), float(scale), _ptr(Y))
    if workspace is None:
        workspace = torch.empty(max(16, e8_gemm_grouped_workspace_bytes(M, K, bpw, len(items))),
                                dtype=torch.uint8, device=X.device)
    _check(load_library().e8_gemm_grouped(cb.handle, _ptr(X), M, int(K), int(bpw),
                                          ctypes.cast(arr, ctypes.c_void_p), len(items),
                                          _ptr(workspace), workspace.numel(), _stream(stream)),
           "e8_gemm_grouped")
    return outs


# ------------------------------------------------------ entropy-coded variant --
class EpMatrix:
    """Compressed form of one matrix (e8_ep_encode): stream words, block
    offsets, row scales t, frequency tables (all on the device)."""

    def __init__(self, N, K, delta, words, offsets, t, tables, total_words):
        self.N, self.K, self.delta = N, K, delta
        self.words, self.offsets, self.t, self.tables = words, offsets, t, tables
        self.total_words = total_words

    def actual_bpp(self) -> float:
        return float(load_library().e8_ep_actual_bpp(self.N, self.K, self.total_words))


def _ep_ws(N, K, dev, workspace):
    return _workspace(load_library().e8_ep_encode_workspace_bytes(N, K), dev, workspace)


def e8_ep_encode(cb: Codebook, W, delta: float, workspace=None, stream=None) -> EpMatrix:
    """W fp32 [N, K] (CUDA) at step delta -> EpMatrix (synchronous)."""
    import torch
    N, K = W.shape
    lib = load_library()
    dev = W.device
    nmax = max(int(lib.e8_ep_max_words(N, K)), 1)
    nb = max(int(lib.e8_ep_num_blocks(N, K)), 0)
    words = torch.empty(nmax, dtype=torch.uint16, device=dev)
    offsets = torch.empty(nb + 1, dtype=torch.int32, device=dev)
    t = torch.empty(max(N, 1), dtype=torch.float32, device=dev)
    tables = torch.empty(E8_EP_TABLE_WORDS, dtype=torch.uint16, device=dev)
    total = ctypes.c_int64(0)
    ws = _ep_ws(N, K, dev, workspace)
    rc = lib.e8_ep_encode(cb.handle, _ptr(W), N, K, float(delta), _ptr(words), nmax,
                          _ptr(offsets), _ptr(t), _ptr(tables), ctypes.byref(total), _ptr(ws),
                          ws.numel(), _stream(stream))
    _check(rc, "e8_ep_encode")
    return EpMatrix(N, K, float(delta), words[:max(total.value, 1)], offsets, t[:N], tables,
                    total.value)


def e8_ep_estimate_bpp(cb: Codebook, W, delta: float, workspace=None, stream=None) -> float:
    N, K = W.shape
    out = ctypes.c_double(0.0)
    ws = _ep_ws(N, K, W.device, workspace)
    rc = load_library().e8_ep_estimate_bpp(cb.handle, _ptr(W), N, K, float(delta),
                                           ctypes.byref(out), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "e8_ep_estimate_bpp")
    return out.value


def e8_ep_choose_delta(cb: Codebook, W, target_bpp: float, workspace=None, stream=None) -> float:
    N, K = W.shape
    out = ctypes.c_float(0.0)
    ws = _ep_ws(N, K, W.device, workspace)
    rc = load_library().e8_ep_choose_delta(cb.handle, _ptr(W), N, K, float(target_bpp),
                                           ctypes.byref(out), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "e8_ep_choose_delta")
    return out.value


def e8_ep_decode_to_bf16(cb: Codebook, m: EpMatrix, out=None, stream=None):
    """bf16 [N, K] weights of an EpMatrix."""
    import torch
    if out is None:
        out = torch.empty((m.N, m.K), dtype=torch.bfloat16, device=m.words.device)
    rc = load_library().e8_ep_decode_to_bf16(cb.handle, _ptr(m.words), m.words.numel(),
                                             _ptr(m.offsets),
                                             _ptr(m.t), _ptr(m.tables), m.N, m.K, _ptr(out),
                                             _stream(stream))
    _check(rc, "e8_ep_decode_to_bf16")
    return out


def e8_ep_gemm(cb: Codebook, X, m: EpMatrix, Y=None, workspace=None, stream=None):
    """Y fp32 [M, N] = X bf16 [M, K] times the decoded weights, transposed."""
    import torch
    M = X.shape[0]
    lib = load_library()
    if Y is None:
        Y = torch.empty((M, m.N), dtype=torch.float32, device=X.device)
    ws = _workspace(lib.e8_ep_gemm_workspace_bytes(M, m.N, m.K), X.device, workspace)
    rc = lib.e8_ep_gemm(cb.handle, _ptr(X), M, _ptr(m.words), m.words.numel(), _ptr(m.offsets),
                        _ptr(m.t),
                        _ptr(m.tables), m.N, m.K, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "e8_ep_gemm")
    return Y



# --------------------------------------------- microscaled 4-bit float form --
class Mx4Matrix:
    """A [rows, K] matrix (or a batch of them) in blocks of 32 e2m1 values with a
    power-of-two scale each, as e8_mx4_encode writes it: codes uint8
    [(batch,) rows, 16 ceil(K / 32)] and scales uint8 [(batch,) bytes in tiles] (other
    one-byte types are taken as their bytes)."""

    __slots__ = ("rows", "K", "batch", "_codes", "_scales", "_both")

    def __init__(self, codes, scales, rows: int, K: int, batch: int | None = None):
        self._codes, self._scales, self._both = codes, scales, None
        self.rows = rows = int(rows)
        self.K = K = int(K)
        self.batch = None if batch is None else int(batch)
        n = 1 if batch is None else self.batch
        # e8_mx4_code_bytes and e8_mx4_scale_bytes
        if codes.element_size() != 1 or scales.element_size() != 1:
            raise E8Error(E8_EINVAL, "Mx4Matrix")
        if rows < 0 or K < 1 or codes.numel() != n * rows * ((K + 31) // 32 * 16) or \
                scales.numel() != n * ((rows + 127) // 128) * ((K + 127) // 128) * 512:
            raise E8Error(E8_EINVAL, "Mx4Matrix")

    @classmethod
    def _new(cls, like, rows, K, batch, stream):
        """Uninitialised, in one tensor: each new tensor costs a call two microseconds, and
        most matrices are handed from one call to the next without a look at the parts."""
        import torch
        m = cls.__new__(cls)
        m.rows, m.K, m.batch, m._codes, m._scales = rows, K, batch, None, None
        at = m._scales_at()
        n = (1 if batch is None else batch) * ((rows + 127) // 128) * ((K + 127) // 128) * 512
        m._both = _mx4_new((at + n,), torch.uint8, like, stream)
        return m

    def _scales_at(self):
        """Place of the scales behind the codes, a multiple of 512 bytes."""
        n = 1 if self.batch is None else self.batch
        return (n * self.rows * ((self.K + 31) // 32 * 16) + 511) // 512 * 512

    def _split(self):
        lead = () if self.batch is None else (self.batch,)
        row = (self.K + 31) // 32 * 16
        n = (1 if self.batch is None else self.batch) * self.rows * row
        self._codes = self._both[:n].view(lead + (self.rows, row))
        self._scales = self._both[self._scales_at():].view(
            lead + (((self.rows + 127) // 128) * ((self.K + 127) // 128) * 512,))

    @property
    def codes(self):
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self):
        if self._codes is None:
            self._split()
        return self._scales

    def _pointers(self, cb, where):
        both = self._both
        if both is not None:
            if both.get_device() != cb.device:
                raise E8Error(E8_EDEVICE, where)
            at = both.data_ptr()
            return at, at + self._scales_at()
        _mx4_check(cb, where, self._codes, self._scales)
        return self._codes.data_ptr(), self._scales.data_ptr()

    def _like(self):
        return self._codes if self._both is None else self._both


_mx4_dtypes = {}


def _mx4_dtype(X) -> int:
    if not _mx4_dtypes:
        import torch
        _mx4_dtypes.update({torch.bfloat16: E8_DT_BF16, torch.float16: E8_DT_F16,
                            torch.float32: E8_DT_F32})
    return _mx4_dtypes.get(X.dtype, -1)


def _mx4_check(cb: Codebook, where: str, *tensors):
    """Device tensors of the codebook's device, densely laid out."""
    dev = cb.device
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise E8Error(E8_EDEVICE, where)
            if not t.is_contiguous():
                raise E8Error(E8_EINVAL, where)


def _mx4_new(shape, dtype, like, stream):
    """A new tensor that belongs to the stream that will write it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _mx4_out(out, shape, dtype, where):
    if out.shape != shape or out.dtype != dtype:
        raise E8Error(E8_EINVAL, where)


def _mx4_stream(cb: Codebook, stream):
    import torch
    return torch._C._cuda_getCurrentRawStream(cb.device) if stream is None else stream.cuda_stream


def _mx4_row_stride(cb: Codebook, X, where: str) -> int:
    if X.get_device() != cb.device:
        raise E8Error(E8_EDEVICE, where)
    if X.is_contiguous():
        return X.shape[-1]
    rows, K = X.shape[-2:]
    if K > 1 and X.stride(-1) != 1:
        raise E8Error(E8_EINVAL, where)
    return K if rows == 1 else X.stride(-2)


@functools.lru_cache(maxsize=1024)
def _mx4_ws_bytes(call: str, *args) -> int:
    return getattr(load_library(), call)(*args)


def e8_mx4_encode(cb: Codebook, X, out: Mx4Matrix | None = None, stream=None) -> Mx4Matrix:
    """X bf16 / fp16 / fp32 [rows, K] or [batch, rows, K] (CUDA) -> Mx4Matrix.

    The last dimension must be dense; rows may be further apart (a slice of a wider
    matrix), matrices rows * row stride apart."""
    import torch
    where = "e8_mx4_encode"
    shape = X.shape
    if len(shape) == 2:
        batch, n = None, 1
        rows, K = shape
    elif len(shape) == 3:
        batch, rows, K = shape
        n = batch
    else:
        raise E8Error(E8_EINVAL, where)
    ldx = _mx4_row_stride(cb, X, where)
    if n > 1 and rows > 0:
        if rows == 1:
            ldx = X.stride(0)
        elif X.stride(0) != rows * ldx:
            raise E8Error(E8_EINVAL, where)
    if out is None:
        if K < 1:
            raise E8Error(E8_EINVAL, where)
        out = Mx4Matrix._new(X, rows, K, batch, stream)
    elif (out.rows, out.K, out.batch) != (rows, K, batch):
        raise E8Error(E8_EINVAL, where)
    codes, scales = out._pointers(cb, where)
    rc = (_lib or load_library()).e8_mx4_encode(
        cb.handle, X.data_ptr(), _mx4_dtype(X), n, rows, K, ldx, codes, scales,
        _mx4_stream(cb, stream))
    if rc:
        _check(rc, where)
    return out


def e8_mx4_decode_to_bf16(cb: Codebook, m: Mx4Matrix, out=None, stream=None):
    """bf16 [(batch,) rows, K] values of an Mx4Matrix."""
    import torch
    where = "e8_mx4_decode_to_bf16"
    shape = (m.rows, m.K) if m.batch is None else (m.batch, m.rows, m.K)
    codes, scales = m._pointers(cb, where)
    if out is None:
        out = _mx4_new(shape, torch.bfloat16, m._like(), stream)
    else:
        _mx4_check(cb, where, out)
        _mx4_out(out, shape, torch.bfloat16, where)
    rc = (_lib or load_library()).e8_mx4_decode_to_bf16(
        cb.handle, codes, scales, 1 if m.batch is None else m.batch, m.rows, m.K, out.data_ptr(),
        _mx4_stream(cb, stream))
    if rc:
        _check(rc, where)
    return out


def e8_mx4_gemm(cb: Codebook, X, m: Mx4Matrix, Y=None, workspace=None, stream=None):
    """Y bf16 [M, N] = X [M, K] (bf16, fp16 or fp32, encoded on the way) times m transposed."""
    import torch
    where = "e8_mx4_gemm"
    shape = X.shape
    if len(shape) != 2 or shape[1] != m.K or m.batch is not None:
        raise E8Error(E8_EINVAL, where)
    M, N, K = shape[0], m.rows, m.K
    ldx = _mx4_row_stride(cb, X, where)
    codes, scales = m._pointers(cb, where)
    _mx4_check(cb, where, Y, workspace)
    if Y is None:
        Y = _mx4_new((M, N), torch.bfloat16, X, stream)
    else:
        _mx4_out(Y, (M, N), torch.bfloat16, where)
    if workspace is None:
        workspace = _mx4_new((_mx4_ws_bytes("e8_mx4_gemm_workspace_bytes", M, N, K),), torch.uint8,
                             X, stream)
    rc = (_lib or load_library()).e8_mx4_gemm(
        cb.handle, X.data_ptr(), _mx4_dtype(X), M, ldx, codes, scales, N, K, Y.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _mx4_stream(cb, stream))
    if rc:
        _check(rc, where)
    return Y


def e8_mx4_gemm_codes(cb: Codebook, a: Mx4Matrix, m: Mx4Matrix, Y=None, workspace=None, stream=None):
    """Y bf16 [M, N] = a [M, K] times m [N, K] transposed, both encoded (no workspace needed)."""
    import torch
    where = "e8_mx4_gemm_codes"
    if a.K != m.K or a.batch is not None or m.batch is not None:
        raise E8Error(E8_EINVAL, where)
    a_codes, a_scales = a._pointers(cb, where)
    codes, scales = m._pointers(cb, where)
    _mx4_check(cb, where, Y, workspace)
    if Y is None:
        Y = _mx4_new((a.rows, m.rows), torch.bfloat16, a._like(), stream)
    else:
        _mx4_out(Y, (a.rows, m.rows), torch.bfloat16, where)
    rc = (_lib or load_library()).e8_mx4_gemm_codes(
        cb.handle, a_codes, a_scales, a.rows, codes, scales, m.rows, m.K, Y.data_ptr(),
        _ptr(workspace),
        0 if workspace is None else workspace.numel(), _mx4_stream(cb, stream))
    if rc:
        _check(rc, where)
    return Y


def e8_mx4_moe(cb: Codebook, X, router, w13: Mx4Matrix, w2: Mx4Matrix, topk: int,
               renormalize: bool = True, Y=None, experts=None, probs=None, workspace=None,
               stream=None):
    """Y bf16 [T, H] of a mixture-of-experts layer for T <= 64 tokens.

    X bf16 [T, H]; router bf16 [E, H]; w13: E matrices [2 I, H] whose even rows are
    the gate's and odd rows the up-projection's; w2: E matrices [H, I].  experts
    (int32 [T, topk]) and probs (fp32 [T, topk]) are filled when given.  All tensors are
    contiguous and start on 16 bytes."""
    import torch
    where = "e8_mx4_moe"
    bf16 = torch.bfloat16
    shape, E, inner, topk = X.shape, w13.batch, w2.K, int(topk)
    if len(shape) != 2 or X.dtype != bf16 or router.dtype != bf16 or E is None:
        raise E8Error(E8_EINVAL, where)
    T, H = shape
    if router.shape != (E, H) or w2.batch != E or w13.rows != 2 * inner or w13.K != H or \
            w2.rows != H:
        raise E8Error(E8_EINVAL, where)
    if experts is not None:
        _mx4_out(experts, (T, topk), torch.int32, where)
    if probs is not None:
        _mx4_out(probs, (T, topk), torch.float32, where)
    codes13, scales13 = w13._pointers(cb, where)
    codes2, scales2 = w2._pointers(cb, where)
    _mx4_check(cb, where, X, router, Y, experts, probs, workspace)
    if Y is None:
        Y = _mx4_new(shape, bf16, X, stream)
    else:
        _mx4_out(Y, shape, bf16, where)
    if workspace is None:
        workspace = _mx4_new((_mx4_ws_bytes("e8_mx4_moe_workspace_bytes", T, H, E, topk, inner),),
                             torch.uint8, X, stream)
    rc = (_lib or load_library()).e8_mx4_moe(
        cb.handle, X.data_ptr(), T, H, router.data_ptr(), E, topk, 1 if renormalize else 0,
        codes13, scales13, inner, codes2, scales2, Y.data_ptr(), _ptr(experts), _ptr(probs),
        workspace.data_ptr(), workspace.numel(), _mx4_stream(cb, stream))
    if rc:
        _check(rc, where)
    return Y


def e8_mx4_moe_pack(cb: Codebook, gate, up, down):
    """Expert weights gate, up [E, I, H] and down [E, H, I] (bf16, fp16 or fp32, CUDA) ->
    (w13, w2) of e8_mx4_moe: gate and up rows interleaved, then encoded."""
    import torch
    if gate.dim() != 3 or gate.shape != up.shape or \
            tuple(down.shape) != (gate.shape[0], gate.shape[2], gate.shape[1]):
        raise E8Error(E8_EINVAL, "e8_mx4_moe_pack")
    both = torch.stack((gate, up), 2).flatten(1, 2)
    return e8_mx4_encode(cb, both), e8_mx4_encode(cb, down.contiguous())
