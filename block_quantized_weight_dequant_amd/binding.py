"""Thin ctypes binding over libq4.so (the C ABI in include/q4.h).

Each function has the name of its C entry point and only marshals arguments:
tensors become device pointers and byte/element counts, ``stream=None`` becomes
PyTorch's current HIP stream, and a non-zero status becomes a ``Q4Error``.
Every step of the computation runs in the library's HIP kernels. There is no
fallback: if the library is missing this module raises on import.

Arguments that are pointers accept a ``torch.Tensor`` (its ``data_ptr()``), a
plain integer address, or ``None`` (NULL).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4.so")

Q4_OK = 0
Q4_ERR_NULL = 1
Q4_ERR_SHAPE = 2
Q4_ERR_SIZE = 3
Q4_ERR_ALIGN = 4
Q4_ERR_ALIAS = 5
Q4_ERR_LAUNCH = 6
Q4_ERR_WORKSPACE = 7
Q4_GEMV_MAX_ROWS = 8
Q4_GEMM_SCRATCH_BYTES = 64 << 20
Q4_MAX_EXPERTS = 1024
Q4_MAX_TOP_K = 32
Q4_MAX_SLOTS = 1 << 30
Q4_NORM_MAX_K = 32768
Q4_ROUTE_MAX_GROUPS = 64
Q4_ACT_SILU = 0
Q4_ACT_GELU = 1
Q4_SCORE_SOFTMAX = 0
Q4_SCORE_SIGMOID = 1
SIZE_MAX = 2 ** 64 - 1

#: Every symbol include/q4.h declares.
EXPORTS = ("q4_abi_version", "q4_status_string", "q4_dequant", "q4_gemv", "q4_gemm",
           "q4_gemm_ws", "q4_gemm_workspace_bytes", "q8_dequant", "q8_gemv", "q8_gemm", "q8_gemm_ws",
           "q8_gemm_workspace_bytes", "q8_quantize", "q4_quantize", "q4_gemm_bf16",
           "q4_gemm_bf16_workspace_bytes", "q8_gemm_bf16", "q8_gemm_bf16_workspace_bytes",
           "q4_gemv_bf16", "q8_gemv_bf16", "q4_gemv_splitk", "q4_gemv_splitk_workspace_bytes",
           "q8_gemv_splitk", "q8_gemv_splitk_workspace_bytes", "q4_gemv_prepare_bytes",
           "q4_gemv_prepare", "q4_gemv_prepared", "q8_gemv_prepare_bytes", "q8_gemv_prepare",
           "q8_gemv_prepared", "q4_gemv_q8a", "q8_gemv_q8a", "q4_gemm_q8a",
           "q4_gemm_q8a_workspace_bytes", "q8_gemm_q8a", "q8_gemm_q8a_workspace_bytes",
           "q4_route", "q4_route_workspace_bytes", "q4_route_groups") + tuple(
               f + "_gemm_grouped" + act + ws for f in ("q4", "q8") for act in ("", "_bf16")
               for ws in ("", "_workspace_bytes")) + tuple(
               f + op + act for f in ("q4", "q8") for op in ("_norm", "_act") for act in ("", "_bf16"))

#: Every symbol include/f8.h declares.
F8_EXPORTS = ("f8_quantize", "f8_quantize_bf16", "f8_dequant", "f8_gemm", "f8_gemv",
              "f8_gemm_grouped", "f8_norm", "f8_norm_bf16", "f8_act", "f8_act_bf16")
F8_BLOCK = 128
F8_MAX_K = 4194304


class Q4Error(RuntimeError):
    def __init__(self, status: int, entry: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (entry, q4_status_string(status), status))


def _load_library():
    # The caller's tensors and streams belong to PyTorch's HIP runtime, and
    # PyTorch ships its own copy of it. Importing torch first makes the dynamic
    # loader resolve libq4.so's libamdhip64.so.7 to that already-loaded copy
    # (same soname); loaded the other way round, the process would hold two
    # HIP runtimes and PyTorch's stream handles would be foreign to ours.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError("libq4.so is not built (%s); run "
                          "`python -m block_quantized_weight_dequant_amd.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.q4_abi_version.restype = i32
    lib.q4_abi_version.argtypes = []
    lib.q4_status_string.restype = ctypes.c_char_p
    lib.q4_status_string.argtypes = [i32]
    for f in ("q4", "q8"):
        getattr(lib, f + "_dequant").restype = i32
        getattr(lib, f + "_dequant").argtypes = [P, sz, P, sz, P]
        for g in ("_gemv", "_gemv_bf16", "_gemm"):
            getattr(lib, f + g).restype = i32
            getattr(lib, f + g).argtypes = [P, P, sz, P, i32, i32, i32, P]
        for g in ("_gemm_ws", "_gemm_bf16"):
            getattr(lib, f + g).restype = i32
            getattr(lib, f + g).argtypes = [P, P, sz, P, i32, i32, i32, P, sz, P]
        for g in ("_gemm_workspace_bytes", "_gemm_bf16_workspace_bytes"):
            getattr(lib, f + g).restype = sz
            getattr(lib, f + g).argtypes = [i32, i32, i32]
        getattr(lib, f + "_gemv_splitk").restype = i32
        getattr(lib, f + "_gemv_splitk").argtypes = [P, P, sz, P, i32, i32, i32, i32, P, sz, P]
        getattr(lib, f + "_gemv_splitk_workspace_bytes").restype = sz
        getattr(lib, f + "_gemv_splitk_workspace_bytes").argtypes = [i32, i32, i32, i32]
        getattr(lib, f + "_gemv_prepare_bytes").restype = sz
        getattr(lib, f + "_gemv_prepare_bytes").argtypes = [i32, i32]
        getattr(lib, f + "_gemv_prepare").restype = i32
        getattr(lib, f + "_gemv_prepare").argtypes = [P, i32, i32, P, sz, P]
        getattr(lib, f + "_gemv_prepared").restype = i32
        getattr(lib, f + "_gemv_prepared").argtypes = [P, sz, P, sz, P, i32, i32, i32, P]
    for name in ("q4_gemv_q8a", "q8_gemv_q8a"):
        getattr(lib, name).restype = i32
        getattr(lib, name).argtypes = [P, sz, P, sz, P, i32, i32, i32, P]
    for name in ("q4_gemm_q8a", "q8_gemm_q8a"):
        getattr(lib, name).restype = i32
        getattr(lib, name).argtypes = [P, sz, P, sz, P, i32, i32, i32, P, sz, P]
        getattr(lib, name + "_workspace_bytes").restype = sz
        getattr(lib, name + "_workspace_bytes").argtypes = [i32, i32, i32]
    for name in ("q8_quantize", "q4_quantize"):
        getattr(lib, name).restype = i32
        getattr(lib, name).argtypes = [P, sz, P, sz, P]
    lib.q4_route.restype = i32
    lib.q4_route.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, sz, P]
    lib.q4_route_workspace_bytes.restype = sz
    lib.q4_route_workspace_bytes.argtypes = [i32, i32, i32]
    for name in ("q4_gemm_grouped", "q4_gemm_grouped_bf16", "q8_gemm_grouped",
                 "q8_gemm_grouped_bf16"):
        getattr(lib, name).restype = i32
        getattr(lib, name).argtypes = [P, P, sz, P, P, i32, P, i32, i32, i32, i32, P, sz, P]
        getattr(lib, name + "_workspace_bytes").restype = sz
        getattr(lib, name + "_workspace_bytes").argtypes = [i32, i32, i32, i32]
    f32 = ctypes.c_float
    lib.q4_route_groups.restype = i32
    lib.q4_route_groups.argtypes = [P, P] + [i32] * 8 + [f32, P, P, P, P, P, sz, P]
    for act in ("", "_bf16"):
        for op, head in (("_norm", [P, P, i32, P, P, P, f32]), ("_act", [P, P, i32, i32])):
            extra = [P] if op == "_norm" else []
            getattr(lib, "q4" + op + act).restype = getattr(lib, "q8" + op + act).restype = i32
            getattr(lib, "q4" + op + act).argtypes = head + [P, i32, i32, i32, P]
            getattr(lib, "q8" + op + act).argtypes = head + extra + [P, sz, i32, i32, P]
            getattr(lib, "f8" + op + act).argtypes = head + extra + [P, sz, P, sz, i32, i32, P]
    for name in F8_EXPORTS:
        getattr(lib, name).restype = i32
    lib.f8_quantize.argtypes = lib.f8_quantize_bf16.argtypes = [P, i32, i32, i32, P, sz, P, sz, P]
    lib.f8_dequant.argtypes = [P, sz, P, sz, i32, i32, i32, P, sz, P]
    lib.f8_gemm.argtypes = lib.f8_gemv.argtypes = [P, P, P, sz, P, P, i32, i32, i32, P]
    lib.f8_gemm_grouped.argtypes = [P, P, P, sz, P, P, P, i32, P, i32, i32, i32, i32, P]
    return lib


lib = _load_library()

import torch  # noqa: E402  (loaded above, before libq4.so)


def _addr(x) -> int:
    """Device address of a tensor argument (an int is taken as an address).
    Host tensors are refused here: the kernels would fault on a host pointer."""
    if x is None:
        return 0
    if getattr(x, "is_cuda", False):
        return x.data_ptr()
    if isinstance(x, int):
        return x
    raise ValueError("expected a device (cuda) tensor, got one on %s" % getattr(x, "device", type(x)))


def _nbytes(x) -> int:
    return x.nbytes


def _stream(stream) -> int:
    if stream is None:
        # Before PyTorch has initialised the GPU its current stream is the
        # default one. The raw handle costs 0.2 us a call, against 3.5 us
        # through a torch.cuda.Stream object.
        if not torch.cuda.is_initialized():
            return 0
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int, entry: str) -> None:
    if status != Q4_OK:
        raise Q4Error(status, entry)


def q4_abi_version() -> int:
    return int(lib.q4_abi_version())


def q4_status_string(status: int) -> str:
    return lib.q4_status_string(int(status)).decode()


def _dequant(entry, w_q, out, w_bytes, out_elems, stream) -> None:
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    oe = int(out.numel()) if out_elems is None else int(out_elems)
    _check(getattr(lib, entry)(_addr(w_q), wb, _addr(out), oe, _stream(stream)), entry)


def q4_dequant(w_q, out, w_bytes=None, out_elems=None, stream=None) -> None:
    """Q4_0 blocks (uint8 tensor) -> f32 ``out``; sizes default to the tensors'."""
    _dequant("q4_dequant", w_q, out, w_bytes, out_elems, stream)


def q8_dequant(w_q, out, w_bytes=None, out_elems=None, stream=None) -> None:
    """Q8_0 blocks (uint8 tensor) -> f32 ``out``; sizes default to the tensors'."""
    _dequant("q8_dequant", w_q, out, w_bytes, out_elems, stream)


def _gemv(entry, a, w_q, y, M, N, K, w_bytes, stream) -> None:
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    _check(getattr(lib, entry)(_addr(a), _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               _stream(stream)), entry)


def q4_gemv(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """y[M, N] = a[M, K] @ dequant(W[N, K/32])^T for 1 <= M <= 8, W Q4_0."""
    _gemv("q4_gemv", a, w_q, y, M, N, K, w_bytes, stream)


def q8_gemv(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """y[M, N] = a[M, K] @ dequant(W[N, K/32])^T for 1 <= M <= 8, W Q8_0."""
    _gemv("q8_gemv", a, w_q, y, M, N, K, w_bytes, stream)


def q4_gemv_bf16(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """As q4_gemv with ``a`` a [M, K] bfloat16 tensor (or its address)."""
    _gemv("q4_gemv_bf16", a, w_q, y, M, N, K, w_bytes, stream)


def q8_gemv_bf16(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """As q8_gemv with ``a`` a [M, K] bfloat16 tensor (or its address)."""
    _gemv("q8_gemv_bf16", a, w_q, y, M, N, K, w_bytes, stream)


def q4_gemv_prepare_bytes(M: int, K: int) -> int:
    return int(lib.q4_gemv_prepare_bytes(int(M), int(K)))


def q8_gemv_prepare_bytes(M: int, K: int) -> int:
    return int(lib.q8_gemv_prepare_bytes(int(M), int(K)))


def _gemv_prepare(entry, a, M, K, prep, prep_bytes, stream) -> None:
    pb = _nbytes(prep) if prep_bytes is None else int(prep_bytes)
    _check(getattr(lib, entry)(_addr(a), int(M), int(K), _addr(prep), pb, _stream(stream)), entry)


def q4_gemv_prepare(a, M: int, K: int, prep, prep_bytes=None, stream=None) -> None:
    """Prepared operands of the f32 activations ``a`` [M, K] for q4_gemv_prepared."""
    _gemv_prepare("q4_gemv_prepare", a, M, K, prep, prep_bytes, stream)


def q8_gemv_prepare(a, M: int, K: int, prep, prep_bytes=None, stream=None) -> None:
    """As q4_gemv_prepare, for q8_gemv_prepared."""
    _gemv_prepare("q8_gemv_prepare", a, M, K, prep, prep_bytes, stream)


def _gemv_prepared(entry, prep, w_q, y, M, N, K, prep_bytes, w_bytes, stream) -> None:
    pb = _nbytes(prep) if prep_bytes is None else int(prep_bytes)
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    _check(getattr(lib, entry)(_addr(prep), pb, _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               _stream(stream)), entry)


def q4_gemv_prepared(prep, w_q, y, M: int, N: int, K: int, prep_bytes=None, w_bytes=None,
                     stream=None) -> None:
    """y[M, N] = a @ dequant(W)^T from operands made by q4_gemv_prepare."""
    _gemv_prepared("q4_gemv_prepared", prep, w_q, y, M, N, K, prep_bytes, w_bytes, stream)


def q8_gemv_prepared(prep, w_q, y, M: int, N: int, K: int, prep_bytes=None, w_bytes=None,
                     stream=None) -> None:
    """As q4_gemv_prepared over a Q8_0 weight stream."""
    _gemv_prepared("q8_gemv_prepared", prep, w_q, y, M, N, K, prep_bytes, w_bytes, stream)


def _gemv_q8a(entry, a_q, w_q, y, M, N, K, a_bytes, w_bytes, stream) -> None:
    ab = _nbytes(a_q) if a_bytes is None else int(a_bytes)
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    _check(getattr(lib, entry)(_addr(a_q), ab, _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               _stream(stream)), entry)


def q4_gemv_q8a(a_q, w_q, y, M: int, N: int, K: int, a_bytes=None, w_bytes=None,
                stream=None) -> None:
    """y[M, N] = dequant(A_q[M, K/32]) @ dequant(W[N, K/32])^T for 1 <= M <= 8:
    activations as Q8_0 blocks (uint8 tensor, e.g. from q8_quantize), W Q4_0."""
    _gemv_q8a("q4_gemv_q8a", a_q, w_q, y, M, N, K, a_bytes, w_bytes, stream)


def q8_gemv_q8a(a_q, w_q, y, M: int, N: int, K: int, a_bytes=None, w_bytes=None,
                stream=None) -> None:
    """As q4_gemv_q8a over a Q8_0 weight stream."""
    _gemv_q8a("q8_gemv_q8a", a_q, w_q, y, M, N, K, a_bytes, w_bytes, stream)


def q4_gemm_q8a_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q4_gemm_q8a_workspace_bytes(int(M), int(N), int(K)))


def q8_gemm_q8a_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q8_gemm_q8a_workspace_bytes(int(M), int(N), int(K)))


def _gemm_q8a(entry, a_q, w_q, y, M, N, K, workspace, workspace_bytes, a_bytes, w_bytes,
              stream) -> None:
    ab = _nbytes(a_q) if a_bytes is None else int(a_bytes)
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    ws = workspace
    if ws is None:
        need = int(getattr(lib, entry + "_workspace_bytes")(int(M), int(N), int(K)))
        if 0 < need < SIZE_MAX:
            ws = _scratch(need, stream, y)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    _check(getattr(lib, entry)(_addr(a_q), ab, _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               _addr(ws), wsb, _stream(stream)), entry)


def q4_gemm_q8a(a_q, w_q, y, M: int, N: int, K: int, workspace=None, workspace_bytes=None,
                a_bytes=None, w_bytes=None, stream=None) -> None:
    """y[M, N] = dequant(A_q[M, K/32]) @ dequant(W[N, K/32])^T for any M: activations
    as Q8_0 blocks, W Q4_0. The workspace comes from PyTorch's allocator when
    none is passed."""
    _gemm_q8a("q4_gemm_q8a", a_q, w_q, y, M, N, K, workspace, workspace_bytes, a_bytes, w_bytes,
              stream)


def q8_gemm_q8a(a_q, w_q, y, M: int, N: int, K: int, workspace=None, workspace_bytes=None,
                a_bytes=None, w_bytes=None, stream=None) -> None:
    """As q4_gemm_q8a over a Q8_0 weight stream."""
    _gemm_q8a("q8_gemm_q8a", a_q, w_q, y, M, N, K, workspace, workspace_bytes, a_bytes, w_bytes,
              stream)


def q4_gemv_splitk_workspace_bytes(M: int, N: int, K: int, splits: int = 0) -> int:
    return int(lib.q4_gemv_splitk_workspace_bytes(int(M), int(N), int(K), int(splits)))


def q8_gemv_splitk_workspace_bytes(M: int, N: int, K: int, splits: int = 0) -> int:
    return int(lib.q8_gemv_splitk_workspace_bytes(int(M), int(N), int(K), int(splits)))


def _gemv_splitk(entry, a, w_q, y, M, N, K, splits, w_bytes, stream, workspace,
                 workspace_bytes) -> None:
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    ws = workspace
    if ws is None:
        need = int(getattr(lib, entry + "_workspace_bytes")(int(M), int(N), int(K), int(splits)))
        if 0 < need < SIZE_MAX:
            ws = _scratch(need, stream, y)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    _check(getattr(lib, entry)(_addr(a), _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               int(splits), _addr(ws), wsb, _stream(stream)), entry)


def q4_gemv_splitk(a, w_q, y, M: int, N: int, K: int, splits: int = 0, w_bytes=None,
                   stream=None, workspace=None, workspace_bytes=None) -> None:
    """As q4_gemv with K split across workgroups (``splits=0``: the library's
    choice); the partials' workspace is taken from PyTorch's caching allocator
    unless one is passed."""
    _gemv_splitk("q4_gemv_splitk", a, w_q, y, M, N, K, splits, w_bytes, stream, workspace,
                 workspace_bytes)


def q8_gemv_splitk(a, w_q, y, M: int, N: int, K: int, splits: int = 0, w_bytes=None,
                   stream=None, workspace=None, workspace_bytes=None) -> None:
    """As q4_gemv_splitk over a Q8_0 weight stream."""
    _gemv_splitk("q8_gemv_splitk", a, w_q, y, M, N, K, splits, w_bytes, stream, workspace,
                 workspace_bytes)


def q4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q4_gemm_workspace_bytes(int(M), int(N), int(K)))


def q8_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q8_gemm_workspace_bytes(int(M), int(N), int(K)))


def _scratch(nbytes: int, stream, like):
    """A uint8 device tensor of nbytes from PyTorch's caching allocator, marked
    as in use by ``stream`` so that it is not handed out again before the work
    queued there has finished."""
    dev = like.device if hasattr(like, "device") else torch.device("cuda", torch.cuda.current_device())
    t = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if stream is None:
        return t
    if isinstance(stream, torch.cuda.Stream):
        t.record_stream(stream)
    elif isinstance(stream, int) and stream != 0:
        t.record_stream(torch.cuda.ExternalStream(stream, device=dev))
    return t


def q4_gemm_bf16_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q4_gemm_bf16_workspace_bytes(int(M), int(N), int(K)))


def q8_gemm_bf16_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.q8_gemm_bf16_workspace_bytes(int(M), int(N), int(K)))


def _gemm(entry, a, w_q, y, M, N, K, w_bytes, stream, workspace, workspace_bytes,
          ws_entry=None) -> None:
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    ws = workspace
    if ws is None:
        need = int(getattr(lib, ws_entry or entry + "_workspace_bytes")(int(M), int(N), int(K)))
        if 0 < need < SIZE_MAX:
            ws = _scratch(need, stream, y)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    _check(getattr(lib, entry)(_addr(a), _addr(w_q), wb, _addr(y), int(M), int(N), int(K),
                               _addr(ws), wsb, _stream(stream)), entry)


def q4_gemm(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """y[M, N] = a[M, K] @ dequant(W[N, K/32])^T for any M, W Q4_0, with no
    workspace: the library's own device scratch (Q4_GEMM_SCRATCH_BYTES per
    GPU) serves it, so calls that overlap in time on one GPU race."""
    _gemv("q4_gemm", a, w_q, y, M, N, K, w_bytes, stream)


def q8_gemm(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """As q4_gemm, with W a Q8_0 stream (the same scratch)."""
    _gemv("q8_gemm", a, w_q, y, M, N, K, w_bytes, stream)


def q4_gemm_ws(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None, workspace=None,
               workspace_bytes=None) -> None:
    """y[M, N] = a[M, K] @ dequant(W[N, K/32])^T for any M, W Q4_0, with the
    caller's workspace.

    ``workspace=None`` takes a scratch tensor of q4_gemm_workspace_bytes(M, N, K)
    bytes from PyTorch's caching allocator for this call; pass a tensor (or an
    address with ``workspace_bytes``) to reuse one."""
    _gemm("q4_gemm_ws", a, w_q, y, M, N, K, w_bytes, stream, workspace, workspace_bytes,
          "q4_gemm_workspace_bytes")


def q8_gemm_ws(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None, workspace=None,
               workspace_bytes=None) -> None:
    """As q4_gemm_ws, with W a Q8_0 stream (workspace from q8_gemm_workspace_bytes)."""
    _gemm("q8_gemm_ws", a, w_q, y, M, N, K, w_bytes, stream, workspace, workspace_bytes,
          "q8_gemm_workspace_bytes")


def q4_gemm_bf16(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None, workspace=None,
                 workspace_bytes=None) -> None:
    """As q4_gemm_ws with ``a`` a [M, K] bfloat16 tensor (or its address); the
    workspace, from q4_gemm_bf16_workspace_bytes, is always needed."""
    _gemm("q4_gemm_bf16", a, w_q, y, M, N, K, w_bytes, stream, workspace, workspace_bytes)


def q8_gemm_bf16(a, w_q, y, M: int, N: int, K: int, w_bytes=None, stream=None, workspace=None,
                 workspace_bytes=None) -> None:
    """As q4_gemm_bf16, with W a Q8_0 stream."""
    _gemm("q8_gemm_bf16", a, w_q, y, M, N, K, w_bytes, stream, workspace, workspace_bytes)


def q8_quantize(x, out_q, n_elems=None, out_bytes=None, stream=None) -> None:
    """f32 ``x`` -> Q8_0 blocks in the uint8 tensor ``out_q``."""
    n = int(x.numel()) if n_elems is None else int(n_elems)
    ob = _nbytes(out_q) if out_bytes is None else int(out_bytes)
    _check(lib.q8_quantize(_addr(x), n, _addr(out_q), ob, _stream(stream)), "q8_quantize")


def q4_quantize(x, out_q, n_elems=None, out_bytes=None, stream=None) -> None:
    """f32 ``x`` -> Q4_0 blocks in the uint8 tensor ``out_q``."""
    n = int(x.numel()) if n_elems is None else int(n_elems)
    ob = _nbytes(out_q) if out_bytes is None else int(out_bytes)
    _check(lib.q4_quantize(_addr(x), n, _addr(out_q), ob, _stream(stream)), "q4_quantize")


def _f8_quantize(entry, x, q, s, M, K, block_rows, q_bytes, s_elems, stream) -> None:
    qb = _nbytes(q) if q_bytes is None else int(q_bytes)
    se = int(s.numel()) if s_elems is None else int(s_elems)
    _check(getattr(lib, entry)(_addr(x), int(M), int(K), int(block_rows), _addr(q), qb, _addr(s),
                               se, _stream(stream)), entry)


def f8_quantize(x, q, s, M: int, K: int, block_rows: int = 1, q_bytes=None, s_elems=None,
                stream=None) -> None:
    """f32 ``x`` [M, K] -> E4M3 codes ``q`` [M, K] (uint8 or float8_e4m3fn) and f32
    scales ``s``, one per 128 columns of a row (``block_rows=1``, activations)
    or per 128 x 128 tile (``block_rows=128``, weights)."""
    _f8_quantize("f8_quantize", x, q, s, M, K, block_rows, q_bytes, s_elems, stream)


def f8_quantize_bf16(x, q, s, M: int, K: int, block_rows: int = 1, q_bytes=None, s_elems=None,
                     stream=None) -> None:
    """As f8_quantize with ``x`` a [M, K] bfloat16 tensor (or its address)."""
    _f8_quantize("f8_quantize_bf16", x, q, s, M, K, block_rows, q_bytes, s_elems, stream)


def f8_dequant(q, s, out, M: int, K: int, block_rows: int = 1, q_bytes=None, s_elems=None,
               out_elems=None, stream=None) -> None:
    """E4M3 codes and scales -> f32 ``out`` [M, K]."""
    qb = _nbytes(q) if q_bytes is None else int(q_bytes)
    se = int(s.numel()) if s_elems is None else int(s_elems)
    oe = int(out.numel()) if out_elems is None else int(out_elems)
    _check(lib.f8_dequant(_addr(q), qb, _addr(s), se, int(M), int(K), int(block_rows), _addr(out),
                          oe, _stream(stream)), "f8_dequant")


def _f8_product(entry, a, a_s, w, w_s, y, M, N, K, w_bytes, stream) -> None:
    wb = _nbytes(w) if w_bytes is None else int(w_bytes)
    _check(getattr(lib, entry)(_addr(a), _addr(a_s), _addr(w), wb, _addr(w_s), _addr(y), int(M),
                               int(N), int(K), _stream(stream)), entry)


def f8_gemm(a, a_s, w, w_s, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """y[M, N] (bfloat16) = a @ w^T for any M, both in E4M3 with a scale for each
    block of 128: ``a`` [M, K] with ``a_s`` [M, ceil(K/128)], ``w`` [N, K] with
    ``w_s`` [ceil(N/128), ceil(K/128)]."""
    _f8_product("f8_gemm", a, a_s, w, w_s, y, M, N, K, w_bytes, stream)


def f8_gemv(a, a_s, w, w_s, y, M: int, N: int, K: int, w_bytes=None, stream=None) -> None:
    """f8_gemm for 1 <= M <= 8 rows."""
    _f8_product("f8_gemv", a, a_s, w, w_s, y, M, N, K, w_bytes, stream)


def f8_gemm_grouped(a, a_s, w, w_s, offsets, order, y, G: int, M: int, N: int, K: int,
                    share: int = 1, w_bytes=None, stream=None) -> None:
    """f8_gemm grouped by expert: row r of group e is ``a``'s row r // share times
    the e-th of G weight matrices. ``offsets`` [G + 1] and ``order`` [M] (or
    None: sorted rows) are int32 device tensors, as q4_route writes them."""
    wb = _nbytes(w) if w_bytes is None else int(w_bytes)
    _check(lib.f8_gemm_grouped(_addr(a), _addr(a_s), _addr(w), wb, _addr(w_s), _addr(offsets),
                               _addr(order), int(share), _addr(y), int(G), int(M), int(N), int(K),
                               _stream(stream)), "f8_gemm_grouped")


def q4_route_workspace_bytes(T: int, E: int, top_k: int) -> int:
    return int(lib.q4_route_workspace_bytes(int(T), int(E), int(top_k)))


def q4_route(logits, ids, weights, offsets, order, T: int, E: int, top_k: int, renorm: bool = True,
             workspace=None, workspace_bytes=None, stream=None) -> None:
    """Router: f32 ``logits`` [T, E] -> ``ids`` [T, top_k] (int32), ``weights``
    [T, top_k] (f32), and the slots sorted by expert: ``offsets`` [E + 1],
    ``order`` [T * top_k] (int32). The workspace comes from PyTorch's allocator
    when none is passed."""
    ws = workspace
    if ws is None:
        need = int(lib.q4_route_workspace_bytes(int(T), int(E), int(top_k)))
        if need:
            ws = _scratch(need, stream, ids)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    _check(lib.q4_route(_addr(logits), int(T), int(E), int(top_k), int(bool(renorm)), _addr(ids),
                        _addr(weights), _addr(offsets), _addr(order), _addr(ws), wsb,
                        _stream(stream)), "q4_route")


def q4_gemm_grouped_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    return int(lib.q4_gemm_grouped_workspace_bytes(int(G), int(M), int(N), int(K)))


def q4_gemm_grouped_bf16_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    return int(lib.q4_gemm_grouped_bf16_workspace_bytes(int(G), int(M), int(N), int(K)))


def q8_gemm_grouped_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    return int(lib.q8_gemm_grouped_workspace_bytes(int(G), int(M), int(N), int(K)))


def q8_gemm_grouped_bf16_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    return int(lib.q8_gemm_grouped_bf16_workspace_bytes(int(G), int(M), int(N), int(K)))


def _gemm_grouped(entry, a, w_q, offsets, order, y, G, M, N, K, share, workspace, workspace_bytes,
                  w_bytes, stream) -> None:
    wb = _nbytes(w_q) if w_bytes is None else int(w_bytes)
    ws = workspace
    if ws is None:
        need = int(getattr(lib, entry + "_workspace_bytes")(int(G), int(M), int(N), int(K)))
        if 0 < need < SIZE_MAX:
            ws = _scratch(need, stream, y)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    _check(getattr(lib, entry)(_addr(a), _addr(w_q), wb, _addr(offsets), _addr(order), int(share),
                               _addr(y), int(G), int(M), int(N), int(K), _addr(ws), wsb,
                               _stream(stream)), entry)


def q4_gemm_grouped(a, w_q, offsets, order, y, G: int, M: int, N: int, K: int, share: int = 1,
                    workspace=None, workspace_bytes=None, w_bytes=None, stream=None) -> None:
    """Products grouped by expert: y[r] = a[r // share] @ dequant(W[e])^T for the
    rows r of each group e, W of G Q4_0 matrices [N, K/32]. ``offsets`` [G + 1]
    and ``order`` [M] (or None: sorted rows) are int32 device tensors, as
    q4_route writes them; rows of y that no group names are left as they were.
    The workspace comes from PyTorch's allocator when none is passed."""
    _gemm_grouped("q4_gemm_grouped", a, w_q, offsets, order, y, G, M, N, K, share, workspace,
                  workspace_bytes, w_bytes, stream)


def q4_gemm_grouped_bf16(a, w_q, offsets, order, y, G: int, M: int, N: int, K: int, share: int = 1,
                         workspace=None, workspace_bytes=None, w_bytes=None, stream=None) -> None:
    """As q4_gemm_grouped with bfloat16 activations."""
    _gemm_grouped("q4_gemm_grouped_bf16", a, w_q, offsets, order, y, G, M, N, K, share, workspace,
                  workspace_bytes, w_bytes, stream)


def q8_gemm_grouped(a, w_q, offsets, order, y, G: int, M: int, N: int, K: int, share: int = 1,
                    workspace=None, workspace_bytes=None, w_bytes=None, stream=None) -> None:
    """As q4_gemm_grouped over Q8_0 matrices."""
    _gemm_grouped("q8_gemm_grouped", a, w_q, offsets, order, y, G, M, N, K, share, workspace,
                  workspace_bytes, w_bytes, stream)


def q8_gemm_grouped_bf16(a, w_q, offsets, order, y, G: int, M: int, N: int, K: int, share: int = 1,
                         workspace=None, workspace_bytes=None, w_bytes=None, stream=None) -> None:
    """As q4_gemm_grouped_bf16 over Q8_0 matrices."""
    _gemm_grouped("q8_gemm_grouped_bf16", a, w_q, offsets, order, y, G, M, N, K, share, workspace,
                  workspace_bytes, w_bytes, stream)


def q4_route_groups(logits, bias, ids, weights, offsets, order, T: int, E: int, top_k: int,
                    score: int = Q4_SCORE_SIGMOID, n_groups: int = 1, top_groups: int = 1,
                    group_best: int = 1, renorm: bool = True, scale: float = 1.0, workspace=None,
                    workspace_bytes=None, stream=None) -> None:
    """Router with scores, a bias and groups: the top_k experts by s + ``bias``
    (f32 [E], or None) among the best ``top_groups`` of ``n_groups`` groups of
    neighbouring experts, s the sigmoid or softmax scores of ``logits``; weights
    scale * s, over their sum with ``renorm``. Outputs and workspace as q4_route."""
    ws = workspace
    if ws is None:
        need = int(lib.q4_route_workspace_bytes(int(T), int(E), int(top_k)))
        if need:
            ws = _scratch(need, stream, ids)
    if workspace_bytes is not None:
        wsb = int(workspace_bytes)
    else:
        wsb = _nbytes(ws) if ws is not None and not isinstance(ws, int) else 0
    slots, dev = T * top_k, _device_of(logits)
    _check(lib.q4_route_groups(_array(logits, T * E, _F32, dev), _array(bias, E, _F32, dev), T, E, top_k,
                               score, n_groups, top_groups, group_best, bool(renorm), scale,
                               _array(ids, slots, _I32, dev), _array(weights, slots, _F32, dev),
                               _array(offsets, E + 1, _I32, dev), _array(order, slots, _I32, dev),
                               _addr(ws), wsb, _stream_for(stream, dev)), "q4_route_groups")


_F32, _I32 = (torch.float32,), (torch.int32,)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_BYTES = (torch.uint8, torch.int8, torch.float8_e4m3fn)
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _device_of(x) -> int:
    """Index of the device that a call's arrays are on: its first input's (-1 of a
    host tensor, which _array then refuses)."""
    return _current_device() if type(x) is int or x is None else x.get_device()


def _array(x, n: int, dtypes, device: int) -> int:
    """Address of a dense tensor of n elements of one of ``dtypes`` on ``device`` (or
    of None, or of a plain address): the kernels go by the sizes given beside it.
    These checks cost 0.2 us a tensor."""
    if x is None:
        return 0
    if type(x) is int:
        return x
    if x.get_device() == device >= 0 and x.dtype in dtypes and x.numel() == n and x.is_contiguous():
        return x.data_ptr()
    raise ValueError("expected a dense tensor of %d elements of %s on %s, got %s" % (
        n, " or ".join(map(str, dtypes)), "a GPU" if device < 0 else "cuda:%d" % device, _what(x)))


def _what(x) -> str:
    return "%s of %s on %s, strides %s" % (tuple(x.shape), x.dtype, x.device, x.stride())


def _stream_for(stream, device: int) -> int:
    """_stream, where the work is on ``device``: without a ``stream`` that has to be
    the current one, whose stream is taken."""
    if stream is not None:
        return _stream(stream)
    if device != _current_device():
        raise ValueError("the tensors are on cuda:%d, which is not the current device: make it current, "
                         "or pass a stream" % device)
    return _current_stream(device)


def _norm(entry, dtypes, dev, x, gamma, M, K, eps, residual, sum, weights, share, out, stream) -> None:
    """out: the arguments between eps and M."""
    n = M * K
    _check(getattr(lib, entry)(
        _array(x, n * share, dtypes, dev), _array(weights, M * share, _F32, dev), share,
        _array(residual, n, dtypes, dev), _array(sum, n, dtypes, dev), _array(gamma, K, _F32, dev), eps,
        *out, M, K, _stream_for(stream, dev)), entry)


def _values_out(y, n: int, y_bf16, dev):
    """Where f32 or bfloat16 values go, and which of the two: by y's type, or by
    ``y_bf16`` where y is an address."""
    bf16 = bool(y_bf16) if type(y) is int or y is None else y.dtype in _BF16
    return _array(y, n, _BF16 if bf16 else _F32, dev), bf16


def _q8_out(out_q, M, K, dev):
    n = M * (K // 32) * 34
    return _array(out_q, n, _BYTES, dev), n


def _f8_out(q, s, M, K, dev):
    n, ns = M * K, M * -(-K // 128)
    return _array(q, n, _BYTES, dev), n, _array(s, ns, _F32, dev), ns


def q4_norm(x, gamma, y, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
            share: int = 1, y_bf16=False, stream=None) -> None:
    """The residual's addition and the root-mean-square norm: h = ``residual`` +
    sum_j weights[m, j] x[m share + j], written to ``sum`` (which may be
    ``residual``), and ``y`` = h / sqrt(mean(h^2) + eps) * gamma in f32 or
    bfloat16, by y's type (of an address: ``y_bf16``). ``x`` [M * share, K],
    ``residual`` and ``sum`` [M, K] f32; ``weights`` [M, share] as q4_route writes
    them, a weight of 0 leaving its row out; ``gamma`` [K] f32."""
    dev = _device_of(x)
    _norm("q4_norm", _F32, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          _values_out(y, M * K, y_bf16, dev), stream)


def q4_norm_bf16(x, gamma, y, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
                 share: int = 1, y_bf16=False, stream=None) -> None:
    """As q4_norm with ``x``, ``residual`` and ``sum`` in bfloat16."""
    dev = _device_of(x)
    _norm("q4_norm_bf16", _BF16, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          _values_out(y, M * K, y_bf16, dev), stream)


def q8_norm(x, gamma, out_q, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
            share: int = 1, y=None, stream=None) -> None:
    """q4_norm with the result as Q8_0 blocks in the uint8 tensor ``out_q``, and in
    f32 in ``y`` as well where that is given."""
    dev = _device_of(x)
    _norm("q8_norm", _F32, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          (_array(y, M * K, _F32, dev), *_q8_out(out_q, M, K, dev)), stream)


def q8_norm_bf16(x, gamma, out_q, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
                 share: int = 1, y=None, stream=None) -> None:
    """As q8_norm with ``x``, ``residual``, ``sum`` and ``y`` in bfloat16."""
    dev = _device_of(x)
    _norm("q8_norm_bf16", _BF16, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          (_array(y, M * K, _BF16, dev), *_q8_out(out_q, M, K, dev)), stream)


def f8_norm(x, gamma, q, s, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
            share: int = 1, y=None, stream=None) -> None:
    """q4_norm with the result as E4M3 codes ``q`` [M, K] and a scale for each 128
    columns, ``s`` [M, ceil(K / 128)], and in f32 in ``y`` as well where that is
    given."""
    dev = _device_of(x)
    _norm("f8_norm", _F32, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          (_array(y, M * K, _F32, dev), *_f8_out(q, s, M, K, dev)), stream)


def f8_norm_bf16(x, gamma, q, s, M: int, K: int, eps: float, residual=None, sum=None, weights=None,
                 share: int = 1, y=None, stream=None) -> None:
    """As f8_norm with ``x``, ``residual``, ``sum`` and ``y`` in bfloat16."""
    dev = _device_of(x)
    _norm("f8_norm_bf16", _BF16, dev, x, gamma, M, K, eps, residual, sum, weights, share,
          (_array(y, M * K, _BF16, dev), *_f8_out(q, s, M, K, dev)), stream)


def _half(x, M, K, dtypes, device: int) -> int:
    """Address of an [M, K] view whose rows are dense."""
    if x is None:
        return 0
    if type(x) is int:
        return x
    if (x.get_device() == device >= 0 and x.dtype in dtypes and x.shape == (M, K) and x.stride(1) == 1):
        return x.data_ptr()
    raise ValueError("expected an [%d, %d] tensor of %s with dense rows on %s, got %s" % (
        M, K, " or ".join(map(str, dtypes)), "a GPU" if device < 0 else "cuda:%d" % device, _what(x)))


def _act(entry, dtypes, dev, gate, up, M, K, act, out, ld, stream) -> None:
    g, u = _half(gate, M, K, dtypes, dev), _half(up, M, K, dtypes, dev)
    if ld is None:
        ld = K if M <= 1 or gate is None or type(gate) is int else gate.stride(0)
    if M > 1:
        for x in (gate, up):
            if x is not None and type(x) is not int and x.stride(0) != ld:
                raise ValueError("expected rows %d elements apart, got %s" % (ld, _what(x)))
    _check(getattr(lib, entry)(g, u, ld, act, *out, M, K, _stream_for(stream, dev)), entry)


def q4_act(gate, up, y, M: int, K: int, act: int = Q4_ACT_SILU, y_bf16=False, ld=None, stream=None) -> None:
    """The gated activation y = f(gate) * up, f SiLU or GELU (tanh form), in f32 or
    bfloat16 by y's type. ``gate`` and ``up`` are f32 [M, K] views with dense
    rows, the halves of one product's rows or two products' results (of
    addresses: ``ld`` elements a row); ``up`` may be None."""
    dev = _device_of(gate)
    _act("q4_act", _F32, dev, gate, up, M, K, act, _values_out(y, M * K, y_bf16, dev), ld, stream)


def q4_act_bf16(gate, up, y, M: int, K: int, act: int = Q4_ACT_SILU, y_bf16=False, ld=None,
                stream=None) -> None:
    """As q4_act with ``gate`` and ``up`` in bfloat16."""
    dev = _device_of(gate)
    _act("q4_act_bf16", _BF16, dev, gate, up, M, K, act, _values_out(y, M * K, y_bf16, dev), ld, stream)


def q8_act(gate, up, out_q, M: int, K: int, act: int = Q4_ACT_SILU, ld=None, stream=None) -> None:
    """q4_act with the result as Q8_0 blocks in the uint8 tensor ``out_q``."""
    dev = _device_of(gate)
    _act("q8_act", _F32, dev, gate, up, M, K, act, _q8_out(out_q, M, K, dev), ld, stream)


def q8_act_bf16(gate, up, out_q, M: int, K: int, act: int = Q4_ACT_SILU, ld=None, stream=None) -> None:
    """As q8_act with ``gate`` and ``up`` in bfloat16."""
    dev = _device_of(gate)
    _act("q8_act_bf16", _BF16, dev, gate, up, M, K, act, _q8_out(out_q, M, K, dev), ld, stream)


def f8_act(gate, up, q, s, M: int, K: int, act: int = Q4_ACT_SILU, ld=None, stream=None) -> None:
    """q4_act with the result as E4M3 codes ``q`` [M, K] and a scale for each 128
    columns, ``s`` [M, ceil(K / 128)]."""
    dev = _device_of(gate)
    _act("f8_act", _F32, dev, gate, up, M, K, act, _f8_out(q, s, M, K, dev), ld, stream)


def f8_act_bf16(gate, up, q, s, M: int, K: int, act: int = Q4_ACT_SILU, ld=None, stream=None) -> None:
    """As f8_act with ``gate`` and ``up`` in bfloat16."""
    dev = _device_of(gate)
    _act("f8_act_bf16", _BF16, dev, gate, up, M, K, act, _f8_out(q, s, M, K, dev), ld, stream)


def raw_status(entry: str, *args) -> int:
    """Call a C entry point with raw integer arguments and return its status
    (for tests of the argument checks)."""
    return int(getattr(lib, entry)(*args))
