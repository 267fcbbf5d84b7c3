"""Thin Python binding of the C ABI in ``include/fa.h`` (argument marshalling only).

Every step of the computation runs in ``libfa_b200.so``; this module checks
tensor shapes the way the ``validate_attention_inputs`` helper of the
holysheep.ai review does (section "Common Errors and Fixes", error 4: same
batch, heads and head_dim for Q, K, V; same sequence length for K and V),
allocates outputs with PyTorch and passes raw device pointers.  There is no
fallback: without the compiled library, a CUDA tensor or an sm_100 device the
call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os
import struct

import torch

from . import build as _build

_lib = None
_HERE = contextlib.nullcontext()

FA_STATUS = {
    0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_ALIGNMENT",
    4: "FA_ERR_DEVICE", 5: "FA_ERR_LAUNCH", 6: "FA_ERR_TIMEOUT", 7: "FA_ERR_WORKSPACE", 8: "FA_ERR_BOUNDS",
    9: "FA_ERR_PLAN",
}


_SIXTEEN = (torch.bfloat16, torch.float16)
FA_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


class FaProblem(ctypes.Structure):
    """The ``fa_problem`` descriptor of include/fa.h."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int), ("N", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("window", ctypes.c_int), ("dtype", ctypes.c_int)]


class FaDecodeProblem(ctypes.Structure):
    """The ``fa_decode_problem`` descriptor of include/fa.h."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int), ("N_q", ctypes.c_int),
                ("N_kv", ctypes.c_int), ("d", ctypes.c_int), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int), ("window", ctypes.c_int), ("dtype", ctypes.c_int)]


class FaRopeProblem(ctypes.Structure):
    """The ``fa_rope_problem`` descriptor of include/fa.h."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("H_k", ctypes.c_int),
                ("d", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("factor", ctypes.c_float), ("dtype", ctypes.c_int),
                ("pos64", ctypes.c_int), ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3),
                ("q_out_stride", ctypes.c_longlong * 3), ("k_out_stride", ctypes.c_longlong * 3),
                ("pos_stride", ctypes.c_longlong * 2)]


class FaCacheProblem(ctypes.Structure):
    """The ``fa_cache_problem`` descriptor of include/fa.h."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int),
                ("P", ctypes.c_int), ("max_pages", ctypes.c_int), ("page", ctypes.c_int), ("dtype", ctypes.c_int),
                ("quant", ctypes.c_int), ("k_stride", ctypes.c_longlong * 2), ("v_stride", ctypes.c_longlong * 2)]


class FaPagedProblem(ctypes.Structure):
    """The ``fa_paged_problem`` descriptor of include/fa.h."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("max_q", ctypes.c_int), ("P", ctypes.c_int), ("max_pages", ctypes.c_int), ("page", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("window", ctypes.c_int),
                ("dtype", ctypes.c_int), ("quant", ctypes.c_int), ("q_stride", ctypes.c_longlong * 2)]


def _packer(cls):
    """Packs the fields of a descriptor, arrays flat, into its bytes (a ctypes object of nested
    arrays takes microseconds to build)."""
    kinds = {ctypes.c_int: "i", ctypes.c_float: "f"}
    s = struct.Struct("@" + "".join(kinds.get(kind) or f"{kind._length_}q" for _, kind in cls._fields_))
    assert s.size == ctypes.sizeof(cls)

    def pack(*values) -> bytes:
        try:
            return s.pack(*values)
        except struct.error as e:
            raise ValueError(f"{cls.__name__}{values}: {e}") from None
    return pack


_pack_rope, _pack_cache, _pack_paged = map(_packer, (FaRopeProblem, FaCacheProblem, FaPagedProblem))


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        super().__init__(f"{what}: {FA_STATUS.get(int(status), 'FA_ERR_UNKNOWN')} ({int(status)})")


def library_path() -> str:
    """The release library, or the checking build (every kernel bounds-checks its TMA
    coordinates and global indices and reports FA_ERR_BOUNDS) when the environment sets
    FA_B200_CHECKS=1 before the first call."""
    return _build.CHECKS_LIB_PATH if os.environ.get("FA_B200_CHECKS") == "1" else _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded ``libfa_b200.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing; build it with `python -m exact_io_aware_93_b200.build` "
            "(there is no non-CUDA fallback)")
    L = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.fa_abi_version.restype = i
    L.fa_status_string.argtypes = [i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    L.fa_fwd.restype = i
    L.fa_get_status.argtypes = [vp]
    L.fa_get_status.restype = i
    L.fa_get_status_site.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    L.fa_get_status_site.restype = i
    L.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
    L.fa_selftest_wait_timeout.restype = i
    L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    L.fa_bwd_workspace_size.restype = ctypes.c_size_t
    L.fa_fwd_ex.argtypes = [ctypes.POINTER(FaProblem), vp, vp, vp, vp, vp, vp]
    L.fa_fwd_ex.restype = i
    L.fa_bwd_ex.argtypes = [ctypes.POINTER(FaProblem), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                            ctypes.c_size_t, vp]
    L.fa_bwd_ex.restype = i
    L.fa_bwd_workspace_size_ex.argtypes = [ctypes.POINTER(FaProblem)]
    L.fa_bwd_workspace_size_ex.restype = ctypes.c_size_t
    L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                         i, i, i, i, f, i, vp]
    L.fa_bwd.restype = i
    L.fa_fwd_e4m3_scaled.argtypes = [ctypes.POINTER(FaProblem), vp, vp, vp, f, f, f, vp, vp, vp]
    L.fa_fwd_e4m3_scaled.restype = i
    L.fa_decode_workspace_size.argtypes = [ctypes.POINTER(FaDecodeProblem)]
    L.fa_decode_workspace_size.restype = ctypes.c_size_t
    L.fa_decode.argtypes = [ctypes.POINTER(FaDecodeProblem), vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.fa_decode.restype = i
    L.fa_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    L.fa_rope.restype = i
    L.fa_cache_append.argtypes = [vp] + [vp] * 10
    L.fa_cache_append.restype = i
    L.fa_cache_gather.argtypes = [vp] + [vp] * 11
    L.fa_cache_gather.restype = i
    L.fa_paged_workspace_size.argtypes = [vp]
    L.fa_paged_workspace_size.restype = ctypes.c_size_t
    L.fa_paged.argtypes = [vp] + [vp] * 11 + [ctypes.c_size_t, vp]
    L.fa_paged.restype = i
    _lib = L
    return L


def _stream_ptr(t: torch.Tensor) -> int:
    """The current stream of t's device.  (The raw handle: building a Stream object first costs
    microseconds, which count beside kernels of a few.)"""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _on(t: torch.Tensor):
    """Make t's device current for a library call: the library takes its SM count, kernel
    set-up and status word from the current device, and launches on that device's stream."""
    return _HERE if t.get_device() == torch._C._cuda_getDevice() else torch.cuda.device(t.device)


def validate_inputs(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> None:
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, seq_len, num_heads, head_dim], got {tuple(t.shape)}")
        if t.dtype not in FA_DTYPE:
            raise TypeError(f"{name} must be bfloat16, float16 or float8_e4m3fn, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.shape[0] == k.shape[0] == v.shape[0]):
        raise ValueError(f"batch size mismatch: {q.shape[0]}, {k.shape[0]}, {v.shape[0]}")
    if k.shape[2] != v.shape[2] or q.shape[2] % k.shape[2] != 0:
        raise ValueError(f"num heads mismatch: {q.shape[2]}, {k.shape[2]}, {v.shape[2]} (key/value heads "
                         "must match each other and divide the query heads)")
    if k.shape[1] != v.shape[1]:
        raise ValueError(f"key/value sequence length mismatch: {k.shape[1]}, {v.shape[1]}")
    if not (q.shape[3] == k.shape[3] == v.shape[3]):
        raise ValueError(f"head dim mismatch: {q.shape[3]}, {k.shape[3]}, {v.shape[3]}")
    if q.shape[1] != k.shape[1]:
        raise ValueError(f"query and key sequence lengths must match: {q.shape[1]}, {k.shape[1]}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on the same device")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError(f"q, k, v must share one dtype, got {q.dtype}, {k.dtype}, {v.dtype}")


def check_buffer(name: str, t: torch.Tensor, shape, dtype: torch.dtype, device: torch.device) -> None:
    """A caller-supplied output must match exactly: the library writes through its raw pointer,
    so a smaller or misplaced buffer would be written out of bounds."""
    if (not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != dtype
            or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def check_scratch(name: str, t: torch.Tensor, device: torch.device) -> None:
    """A caller-supplied workspace: any dtype, contiguous, on the inputs' device (its byte size
    is checked by the library)."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")


def problem(q: torch.Tensor, k: torch.Tensor, causal: bool, scale: float | None,
            window: int | None) -> FaProblem:
    B, N, H, d = q.shape
    return FaProblem(B, H, k.shape[2], N, d, 1.0 / math.sqrt(d) if scale is None else float(scale),
                     int(bool(causal)), -1 if window is None else int(window), FA_DTYPE[q.dtype])


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
        scale: float | None = None, out: torch.Tensor | None = None,
        lse: torch.Tensor | None = None, window: int | None = None):
    """(O [B, N, H, d] in q's dtype, LSE [B, H, N] fp32) of exact attention via ``fa_fwd_ex``.

    k and v may have fewer heads than q (grouped-query attention); ``window`` (causal only)
    limits query i to keys i - window .. i."""
    validate_inputs(q, k, v)
    B, N, H, d = q.shape
    out_dtype = torch.bfloat16 if q.dtype == torch.float8_e4m3fn else q.dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    check_buffer("out", out, q.shape, out_dtype, q.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    check_buffer("lse", lse, (B, H, N), torch.float32, q.device)
    p = problem(q, k, causal, scale, window)
    with _on(q):
        st = lib().fa_fwd_ex(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                             lse.data_ptr(), _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_fwd_ex")
    return out, lse


def fwd_e4m3(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_descale: float, k_descale: float,
             v_descale: float, causal: bool = False, scale: float | None = None, out: torch.Tensor | None = None,
             lse: torch.Tensor | None = None, window: int | None = None):
    """(O [B, N, H, d] bf16, LSE [B, H, N] fp32) of attention over the values ``codes * descale``
    of fp8 e4m3 inputs (torch.float8_e4m3fn), via ``fa_fwd_e4m3_scaled`` (d = 128)."""
    validate_inputs(q, k, v)
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError("fwd_e4m3 takes float8_e4m3fn codes")
    B, N, H, d = q.shape
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    check_buffer("out", out, q.shape, torch.bfloat16, q.device)
    check_buffer("lse", lse, (B, H, N), torch.float32, q.device)
    p = problem(q, k, causal, scale, window)
    with _on(q):
        st = lib().fa_fwd_e4m3_scaled(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      float(q_descale), float(k_descale), float(v_descale), out.data_ptr(),
                                      lse.data_ptr(), _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_fwd_e4m3_scaled")
    return out, lse


def bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    """Bytes of device workspace ``fa_bwd`` needs (fp32 dQ accumulator and row sums D)."""
    return int(lib().fa_bwd_workspace_size(B, H, N, d))


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, do: torch.Tensor,
        lse: torch.Tensor, causal: bool = False, scale: float | None = None,
        dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
        workspace: torch.Tensor | None = None, window: int | None = None):
    """(dQ, dK, dV) of L = sum(O * dO) via ``fa_bwd_ex`` (score tiles recomputed from LSE)."""
    validate_inputs(q, k, v)
    for name, t in (("o", o), ("do", do)):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous tensor shaped like q, of q's dtype")
    B, N, H, d = q.shape
    check_buffer("lse", lse, (B, H, N), torch.float32, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    check_buffer("dq", dq, q.shape, q.dtype, q.device)
    check_buffer("dk", dk, k.shape, k.dtype, q.device)
    check_buffer("dv", dv, v.shape, v.dtype, q.device)
    p = problem(q, k, causal, scale, window)
    need = int(lib().fa_bwd_workspace_size_ex(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    check_scratch("workspace", workspace, q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    with _on(q):
        st = lib().fa_bwd_ex(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                             workspace.data_ptr(), ws_bytes, _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_bwd_ex")
    return dq, dk, dv


def decode_problem(q: torch.Tensor, k_cache: torch.Tensor, causal: bool, scale: float | None,
                   window: int | None) -> FaDecodeProblem:
    B, n_q, H, d = q.shape
    return FaDecodeProblem(B, H, k_cache.shape[2], n_q, k_cache.shape[1], d,
                           1.0 / math.sqrt(d) if scale is None else float(scale), int(bool(causal)),
                           -1 if window is None else int(window), FA_DTYPE.get(q.dtype, -1))


def decode_workspace_size(q: torch.Tensor, k_cache: torch.Tensor, causal: bool = True,
                          window: int | None = None) -> int:
    """Bytes of device workspace ``fa_decode`` needs for these shapes on q's device (the split
    depends on that device's SM count)."""
    with _on(q):
        return int(lib().fa_decode_workspace_size(ctypes.byref(decode_problem(q, k_cache, causal, None, window))))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           seqlens: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
           out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None, window: int | None = None):
    """(O [B, N_q, H, d] in q's dtype, LSE [B, H, N_q] fp32) of N_q new queries per sequence against a
    key/value cache ``[B, N_kv, H_kv, d]`` via ``fa_decode``.

    ``seqlens`` (int32 [B] on the device, or None for full caches) gives each sequence's cached
    length; with ``causal`` the queries are the last N_q positions of each sequence: query i
    of sequence b stands at position seqlens[b] - N_q + i."""
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4 or t.dtype not in FA_DTYPE or t.dtype != q.dtype:
            raise ValueError(f"{name} must be a 4-d bfloat16 or float16 tensor of q's dtype")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor (no CPU path)")
    B, n_q, H, d = q.shape
    if k_cache.shape != v_cache.shape or k_cache.shape[0] != B or k_cache.shape[3] != d:
        raise ValueError(f"cache shapes {tuple(k_cache.shape)}, {tuple(v_cache.shape)} do not fit q {tuple(q.shape)}")
    if H % k_cache.shape[2] != 0:
        raise ValueError("key/value heads must divide the query heads")
    if not (k_cache.device == v_cache.device == q.device):
        raise ValueError("q, k_cache and v_cache must be on the same device")
    if seqlens is not None:
        check_buffer("seqlens", seqlens, (B,), torch.int32, q.device)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, n_q), dtype=torch.float32, device=q.device) if lse is None else lse
    check_buffer("out", out, q.shape, q.dtype, q.device)
    check_buffer("lse", lse, (B, H, n_q), torch.float32, q.device)
    p = decode_problem(q, k_cache, causal, scale, window)
    with _on(q):
        need = int(lib().fa_decode_workspace_size(ctypes.byref(p)))
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        check_scratch("workspace", workspace, q.device)
        ws_bytes = workspace.numel() * workspace.element_size()
        st = lib().fa_decode(ctypes.byref(p), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             None if seqlens is None else seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(),
                             workspace.data_ptr(), ws_bytes, _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_decode")
    return out, lse


def _check_heads(name: str, t: torch.Tensor, like: torch.Tensor | None = None) -> None:
    """A [.., heads, d] tensor of a 16-bit type on the GPU with contiguous columns (any other
    strides), of ``like``'s type and device."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise ValueError(f"{name} must be [tokens, heads, d] or [batch, seq_len, heads, d]")
    dtype = t.dtype
    if dtype not in _SIXTEEN or (like is not None and dtype != like.dtype):
        raise TypeError(f"{name} must be bfloat16 or float16, one type for all, got {dtype}")
    if not t.is_cuda or (like is not None and t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path), one device for all")
    if t.stride()[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name} must have contiguous columns")


def _span(t: torch.Tensor) -> tuple[int, int]:
    at = t.data_ptr()
    if t.is_contiguous():
        return at, at + t.numel() * t.element_size()
    shape, stride = t.shape, t.stride()
    return at, at + (sum(map(operator.mul, shape, stride)) - sum(stride) + 1) * t.element_size()


def _interleaved(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors whose spans overlap have no element in common all the same, as slices of one
    buffer do: then all of a and all of b lie in two parts of one period, a stride of a, once the
    strides that are multiples of the period are left out."""
    size = a.element_size()
    gap = b.data_ptr() - a.data_ptr()
    if b.element_size() != size or gap % size:
        return False
    gap //= size
    dims = [list(zip(t.shape, t.stride())) for t in (a, b)]
    for period in a.stride()[:-1]:
        if period > 0:
            room, more = [sum([(n - 1) * st for n, st in d if st % period], 1) for d in dims]
            at = gap % period
            if room <= at and at + more <= period:
                return True
    return False


def _spans(*tensors: torch.Tensor | None) -> list[tuple[int, int]]:
    return [_span(t) for t in tensors if t is not None and t.numel()]


def _check_spans(name: str, out: torch.Tensor, spans: list[tuple[int, int]]) -> None:
    """A caller's output that the call would write while it still reads, or writes, one of the others."""
    lo, hi = _span(out)
    for first, end in spans:
        if lo < end and first < hi and out.numel():
            raise ValueError(f"{name} must not overlap the call's other tensors")


def _check_apart(name: str, out: torch.Tensor, *others: torch.Tensor | None) -> None:
    _check_spans(name, out, _spans(*others))


def _check_rope_out(name: str, out: torch.Tensor, x: torch.Tensor, *others: torch.Tensor | None) -> None:
    """An output of rope: x's shape, no element twice, x itself or apart from it (a partial overlap
    would be read after it is written), and apart from the others."""
    if out is not x:
        _check_heads(name, out, x)
        if out.shape != x.shape:
            raise ValueError(f"{name} must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    shape, stride = out.shape, out.stride()
    reach = 1
    for st, n in sorted((st, n) for n, st in zip(shape, stride) if n > 1):
        if st < reach:
            raise ValueError(f"{name} must not overlap itself")
        reach = st * (n - 1) + reach
    lo = out.data_ptr()
    hi = lo + reach * out.element_size()
    if out is not x and (lo != x.data_ptr() or stride != x.stride()):
        others = (x, *others)
    for t in others:
        if t is not None and t.numel() and out.numel():
            first, end = _span(t)
            if lo < end and first < hi and not _interleaved(out, t):
                raise ValueError(f"{name} must be its input itself or lie apart from the inputs and the other output")


def _empty_like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _strides3(t: torch.Tensor):
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


_NO_STRIDES = (0, 0, 0)


def _rope(q, k, positions, inv_freq, interleaved, factor, q_out, k_out, inverse):
    _check_heads("q", q)
    shape, device = q.shape, q.get_device()
    if k is not None:
        _check_heads("k", k, q)
        k_shape = k.shape
        if len(k_shape) != len(shape) or (*k_shape[:-2], shape[-2], k_shape[-1]) != shape:
            raise ValueError(f"k {tuple(k_shape)} does not fit q {tuple(shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    lead, d = shape[:-2], shape[-1]
    if (not isinstance(positions, torch.Tensor) or positions.dtype not in _INTS
            or positions.get_device() != device or (positions.shape != lead and positions.shape != lead[-1:])):
        raise ValueError(f"positions must be int32 or int64 of shape {tuple(lead)} or {tuple(lead[-1:])} on {q.device}")
    if (not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 or inv_freq.dim() != 1
            or inv_freq.get_device() != device or not inv_freq.is_contiguous()
            or not 1 <= inv_freq.numel() <= d // 2):
        raise ValueError(f"inv_freq must be a contiguous float64 vector of 1 to {d // 2} entries on {q.device}")
    given = (q_out, k_out)
    q_out = _empty_like(q) if q_out is None else q_out
    if k is not None and k_out is None:
        k_out = _empty_like(k)
    if given[0] is not None:
        _check_rope_out("q_out", q_out, q, k, None if k_out is k else k_out)
    if given[1] is not None:
        _check_rope_out("k_out", k_out, k, None if q_out is q else q)
    if q.numel() == 0 and (k is None or k.numel() == 0):
        return q_out, k_out
    B, N = (1, shape[0]) if len(shape) == 3 else (shape[0], shape[1])
    pos_stride = positions.stride()
    if k is None:
        k_heads, k_strides, k_out_strides, k_ptr, k_out_ptr = 0, _NO_STRIDES, _NO_STRIDES, None, None
    else:
        k_heads, k_strides, k_out_strides = k_shape[-2], _strides3(k), _strides3(k_out)
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    p = _pack_rope(B, N, shape[-2], k_heads, d, 2 * inv_freq.numel(), 1 if interleaved else 0, 1 if inverse else 0,
                   float(factor), FA_DTYPE[q.dtype], 1 if positions.dtype == torch.int64 else 0, *_strides3(q),
                   *k_strides, *_strides3(q_out), *k_out_strides, pos_stride[0] if len(pos_stride) == 2 else 0,
                   pos_stride[-1])
    with _on(q):
        st = lib().fa_rope(p, q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr, positions.data_ptr(),
                           inv_freq.data_ptr(), _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_rope")
    return q_out, k_out


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
         interleaved: bool = False, factor: float = 1.0, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None):
    """(q, k) rotated by their positions via ``fa_rope``: pair j of the first 2 * len(inv_freq)
    columns of every head turns by position * inv_freq[j] and is scaled by ``factor``; the other
    columns are copied.  The pair is columns (j, j + len(inv_freq)), or (2j, 2j + 1) when
    ``interleaved``.

    q is [T, H, d] or [B, N, H, d] and k the same with its own heads (or None), bfloat16 or
    float16, with any strides but contiguous columns (slices of a fused projection).
    ``positions`` is int32 or int64 of the leading shape, or [N] for every batch row;
    ``inv_freq`` is float64 (``rotary.rope_frequencies``).  An output may be its input itself; apart
    from that, given outputs share no element with each other or with q and k (slices of one buffer
    may interleave)."""
    return _rope(q, k, positions, inv_freq, interleaved, factor, q_out, k_out, False)


def rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
             interleaved: bool = False, factor: float = 1.0, q_grad: torch.Tensor | None = None,
             k_grad: torch.Tensor | None = None):
    """The gradients of ``rope``'s inputs from those of its outputs (the transposed rotation), with
    the arguments of the forward call."""
    return _rope(dq, dk, positions, inv_freq, interleaved, factor, q_grad, k_grad, True)


_SCALE_TYPES = (torch.float8_e8m0fnu, torch.uint8)
_INT32 = (torch.int32,)
_INTS = (torch.int32, torch.int64)


def _is(t, shape, dtypes, device: int) -> bool:
    """A contiguous tensor of this shape, one of these types, on this device."""
    return (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.get_device() == device
            and t.is_contiguous())


def _check_pages(k_pages, v_pages, page_table, seqlens, k_scales, v_scales, dtype) -> bool:
    """The tensors of a paged cache read or written as ``dtype``; True for an e4m3 pool."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if (not isinstance(t, torch.Tensor) or t.dim() != 4 or not t.is_cuda or not t.is_contiguous()
                or t.numel() == 0):
            raise ValueError(f"{name} must be a contiguous CUDA tensor [pages, kv_heads, page, d], none of them 0")
    shape, kind, device = k_pages.shape, k_pages.dtype, k_pages.get_device()
    if v_pages.shape != shape or v_pages.dtype != kind or v_pages.get_device() != device:
        raise ValueError("k_pages and v_pages must have one shape, dtype and device")
    quant = kind == torch.float8_e4m3fn
    if not quant:
        if kind != dtype:
            raise TypeError(f"pages of {kind} do not fit {dtype} (pages are of that type, or float8_e4m3fn)")
        if k_scales is not None or v_scales is not None:
            raise ValueError("scales given for 16-bit pages")
    elif not (_is(k_scales, shape[:3], _SCALE_TYPES, device) and _is(v_scales, shape[:3], _SCALE_TYPES, device)):
        raise ValueError(f"k_scales and v_scales must be contiguous float8_e8m0fnu tensors of shape {tuple(shape[:3])} "
                         f"on {k_pages.device}")
    if (not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.dtype != torch.int32
            or page_table.get_device() != device or not page_table.is_contiguous()):
        raise ValueError(f"page_table must be a contiguous int32 [sequences, pages] tensor on {k_pages.device}")
    if not _is(seqlens, page_table.shape[:1], _INT32, device):
        check_buffer("seqlens", seqlens, (page_table.shape[0],), torch.int32, k_pages.device)
    return quant


def _check_pools(a: torch.Tensor, b: torch.Tensor, *rows) -> None:
    """Pools that are written: apart from each other and from the rows written to them (tensors, or
    spans known already)."""
    nbytes, pa, pb = a.numel() * a.element_size(), a.data_ptr(), b.data_ptr()
    if abs(pa - pb) < nbytes:
        raise ValueError("the pools of keys and values must not overlap")
    for t in rows:
        lo, hi = t if type(t) is tuple else _span(t)
        if lo < hi and (lo < pa + nbytes and pa < hi or lo < pb + nbytes and pb < hi):
            raise ValueError("new keys and values must not lie in the pools")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def cache_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 page_table: torch.Tensor, seqlens: torch.Tensor, cu_q: torch.Tensor,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None) -> None:
    """Write new keys and values [T, H_kv, d] (any strides but contiguous columns and rows aligned to 16
    bytes) into a paged cache via ``fa_cache_append``.

    Sequence b owns rows cu_q[b] .. cu_q[b + 1] (int32 [B + 1]), the last of its seqlens[b]
    positions (int32 [B], the new rows included); rows behind cu_q[B] are not written.  Position p
    lies in page page_table[b, p // page] (int32 [B, max_pages]) at slot p % page of the pools
    [P, H_kv, page, d].  Pools of float8_e4m3fn take codes with one power-of-two scale per row in
    ``k_scales`` / ``v_scales`` (float8_e8m0fnu [P, H_kv, page]).  Everything but the shapes is read
    on the device; bad positions and page numbers skip their row and set the status word.  The pools
    overlap neither each other nor the new rows."""
    for name, t in (("k", k), ("v", v)):
        _check_heads(name, t, k)
        if t.dim() != 3 or t.shape != k.shape:
            raise ValueError(f"{name} must be [tokens, kv_heads, d], k and v of one shape")
    quant = _check_pages(k_pages, v_pages, page_table, seqlens, k_scales, v_scales, k.dtype)
    P, H_kv, page, d = k_pages.shape
    B, max_pages = page_table.shape
    T, heads, width = k.shape
    if k.get_device() != k_pages.get_device() or heads != H_kv or width != d:
        raise ValueError(f"k {tuple(k.shape)} does not fit pages {tuple(k_pages.shape)} on {k_pages.device}")
    if not _is(cu_q, (B + 1,), _INT32, k.get_device()):
        check_buffer("cu_q", cu_q, (B + 1,), torch.int32, k.device)
    if T == 0:
        return
    (k_tok, k_head, _), (v_tok, v_head, _), kp, vp = k.stride(), v.stride(), k.data_ptr(), v.data_ptr()
    rows = ((kp, kp + 2 * ((T - 1) * k_tok + (H_kv - 1) * k_head + d)),
            (vp, vp + 2 * ((T - 1) * v_tok + (H_kv - 1) * v_head + d)))
    _check_pools(k_pages, v_pages, *rows)
    if quant:
        _check_pools(k_scales, v_scales, *rows)
    p = _pack_cache(B, T, H_kv, d, P, max_pages, page, FA_DTYPE[k.dtype], 1 if quant else 0, k_tok, k_head, v_tok, v_head)
    with _on(k):
        st = lib().fa_cache_append(p, kp, vp, k_pages.data_ptr(), v_pages.data_ptr(),
                                   _ptr(k_scales), _ptr(v_scales), page_table.data_ptr(), seqlens.data_ptr(),
                                   cu_q.data_ptr(), _stream_ptr(k))
    if st != 0:
        raise FAError(st, "fa_cache_append")


def cache_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, seqlens: torch.Tensor,
                 cu_k: torch.Tensor, total: int, starts: torch.Tensor | None = None,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
                 dtype: torch.dtype | None = None, k_out: torch.Tensor | None = None,
                 v_out: torch.Tensor | None = None):
    """(k, v) [total, H_kv, d] read back from a paged cache via ``fa_cache_gather``: row cu_k[b] + i is
    position starts[b] + i of sequence b (``starts`` None: from 0).  Rows whose position is at or past
    seqlens[b], and rows behind cu_k[B], are left as they were.  ``dtype`` is the type of the values
    read from e4m3 pages (bfloat16 when not given); 16-bit pages are read as they are.  Given outputs
    overlap neither each other nor what the call reads."""
    if dtype is None:
        is8 = isinstance(k_pages, torch.Tensor) and k_pages.dtype == torch.float8_e4m3fn
        dtype = torch.bfloat16 if is8 or not isinstance(k_pages, torch.Tensor) else k_pages.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    quant = _check_pages(k_pages, v_pages, page_table, seqlens, k_scales, v_scales, dtype)
    P, H_kv, page, d = k_pages.shape
    B, max_pages = page_table.shape
    total = int(total)
    if total < 0:
        raise ValueError(f"total must not be negative, got {total}")
    device = k_pages.get_device()
    if not _is(cu_k, (B + 1,), _INT32, device):
        check_buffer("cu_k", cu_k, (B + 1,), torch.int32, k_pages.device)
    if starts is not None and not _is(starts, (B,), _INT32, device):
        check_buffer("starts", starts, (B,), torch.int32, k_pages.device)
    shape, given = (total, H_kv, d), (k_out, v_out)
    k_out = k_pages.new_empty(shape, dtype=dtype) if k_out is None else k_out
    v_out = k_pages.new_empty(shape, dtype=dtype) if v_out is None else v_out
    for name, out, other in (("k_out", given[0], v_out), ("v_out", given[1], k_out)):
        if out is not None:
            check_buffer(name, out, shape, dtype, k_pages.device)
            _check_apart(name, out, other, k_pages, v_pages, k_scales, v_scales, page_table, seqlens, cu_k, starts)
    if total == 0:
        return k_out, v_out
    p = _pack_cache(B, total, H_kv, d, P, max_pages, page, FA_DTYPE[dtype], 1 if quant else 0, 0, 0, 0, 0)
    with _on(k_pages):
        st = lib().fa_cache_gather(p, k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales),
                                   _ptr(v_scales), page_table.data_ptr(), seqlens.data_ptr(), cu_k.data_ptr(),
                                   _ptr(starts), k_out.data_ptr(), v_out.data_ptr(), _stream_ptr(k_pages))
    if st != 0:
        raise FAError(st, "fa_cache_gather")
    return k_out, v_out


def _paged_problem(q, k_pages, page_table, max_q, causal, scale, window, quant) -> bytes:
    T, H, d = q.shape
    P, H_kv, page, _ = k_pages.shape
    B, max_pages = page_table.shape
    stride = q.stride()
    return _pack_paged(B, T, H, H_kv, int(max_q), P, max_pages, page, d,
                       1.0 / math.sqrt(d) if scale is None else float(scale), 1 if causal else 0,
                       -1 if window is None else int(window), FA_DTYPE[q.dtype], 1 if quant else 0, stride[0], stride[1])


def paged_workspace_size(q: torch.Tensor, k_pages: torch.Tensor, page_table: torch.Tensor, max_q: int) -> int:
    """Bytes of device workspace ``fa_paged`` needs for these shapes on q's device."""
    quant = k_pages.dtype == torch.float8_e4m3fn
    p = _paged_problem(q, k_pages, page_table, max_q, True, None, None, quant)
    with _on(q):
        return int(lib().fa_paged_workspace_size(p))


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                    seqlens: torch.Tensor, cu_q: torch.Tensor, max_q: int, causal: bool = True,
                    scale: float | None = None, window: int | None = None, k_scales: torch.Tensor | None = None,
                    v_scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(O [T, H, d] in q's dtype, LSE [H, T] fp32) of the new tokens of a ragged batch against their
    paged caches (``cache_append``'s layout), via ``fa_paged``.

    Sequence b owns tokens cu_q[b] .. cu_q[b + 1] of q [T, H, d] (at most ``max_q``, any strides but
    contiguous columns and rows aligned to 16 bytes): one token (decoding), a few (drafted tokens) or a
    chunk of a prompt, mixed freely.  With ``causal`` its token i stands at position seqlens[b] - n_b + i and sees the keys at
    or before it, with ``window`` no more than that many back; without, all seqlens[b] keys.  A token
    that sees no key gets O = 0 and LSE = -inf; rows behind cu_q[B] are left as they were.  Given
    outputs and a given workspace (``paged_workspace_size`` bytes, for calls that do not overlap in time)
    lie apart from what the call reads and from each other."""
    _check_heads("q", q)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, d]")
    quant = _check_pages(k_pages, v_pages, page_table, seqlens, k_scales, v_scales, q.dtype)
    T, H, d = q.shape
    device = q.get_device()
    if device != k_pages.get_device() or d != k_pages.shape[3] or H % k_pages.shape[1] != 0:
        raise ValueError(f"q {tuple(q.shape)} does not fit pages {tuple(k_pages.shape)} on {k_pages.device} "
                         "(key/value heads must divide the query heads)")
    if not _is(cu_q, (page_table.shape[0] + 1,), _INT32, device):
        check_buffer("cu_q", cu_q, (page_table.shape[0] + 1,), torch.int32, q.device)
    spans = None
    if out is not None or lse is not None or workspace is not None:
        spans = _spans(q, k_pages, v_pages, k_scales, v_scales, page_table, seqlens, cu_q)
    if out is None:
        out = _empty_like(q)
    else:
        check_buffer("out", out, q.shape, q.dtype, q.device)
        _check_spans("out", out, spans)
    if lse is None:
        lse = q.new_empty((H, T), dtype=torch.float32)
    else:
        check_buffer("lse", lse, (H, T), torch.float32, q.device)
        _check_spans("lse", lse, spans + [_span(out)])
    if T == 0:
        return out, lse
    p = _paged_problem(q, k_pages, page_table, max_q, causal, scale, window, quant)
    with _on(q):
        if workspace is None:
            need = int(lib().fa_paged_workspace_size(p))
            workspace = q.new_empty(max(need, 1), dtype=torch.uint8)
        else:
            check_scratch("workspace", workspace, q.device)
            _check_spans("workspace", workspace, spans + [_span(out), _span(lse)])
        st = lib().fa_paged(p, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales),
                            _ptr(v_scales), page_table.data_ptr(), seqlens.data_ptr(), cu_q.data_ptr(),
                            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream_ptr(q))
    if st != 0:
        raise FAError(st, "fa_paged")
    return out, lse


def get_status(device: torch.device | None = None) -> int:
    """Synchronise the device's current stream and read-and-clear that device's status word
    (the current device when none is given)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev)
        return int(lib().fa_get_status(ctypes.c_void_p(s.cuda_stream)))


def get_status_site(device: torch.device | None = None) -> tuple[int, int]:
    """As get_status, and also where the first recorded error arose: the site number of the
    wait that ran out or of the bounds check that failed (0 when none was recorded)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    site = ctypes.c_int(0)
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev)
        st = int(lib().fa_get_status_site(ctypes.c_void_p(s.cuda_stream), ctypes.byref(site)))
    return st, int(site.value)


def selftest_wait_timeout(timeout_us: int = 20000) -> int:
    """Run the bounded-wait self-test on the current stream; returns the launch status."""
    s = torch.cuda.current_stream()
    return int(lib().fa_selftest_wait_timeout(int(timeout_us), ctypes.c_void_p(s.cuda_stream)))


def attention(q, k, v, causal: bool = False, scale: float | None = None) -> torch.Tensor:
    """O only."""
    return fwd(q, k, v, causal=causal, scale=scale)[0]
