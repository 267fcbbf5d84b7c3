"""Refusals of the paged attention entry points: documented codes, before any device work."""
import ctypes

import pytest
import torch

from exact_io_aware_93_b200 import build as fabuild
from exact_io_aware_93_b200.api import FaPagedProblem

P = 0x10000
NO_GPU = not torch.cuda.is_available()
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(fabuild.build())
    L.fa_paged.argtypes = [ctypes.POINTER(FaPagedProblem)] + [vp] * 11 + [ctypes.c_size_t, vp]
    L.fa_paged_workspace_size.argtypes = [ctypes.POINTER(FaPagedProblem)]
    L.fa_paged_workspace_size.restype = ctypes.c_size_t
    return L


def problem(**kw):
    base = dict(B=2, T=5, H=4, H_kv=2, max_q=3, P=9, max_pages=4, page=16, d=64, scale=0.125, causal=1, window=-1,
                dtype=0, quant=0, q_stride=(256, 64))
    base.update(kw)
    return ctypes.byref(FaPagedProblem(**base))


def call(lib, q=P, kp=P, v=P, ks=0, vs=0, table=P, lens=P, cu=P, o=P, lse=P, ws=P, ws_bytes=0, **kw):
    return lib.fa_paged(problem(**kw), vp(q), vp(kp), vp(v), vp(ks), vp(vs), vp(table), vp(lens), vp(cu), vp(o), vp(lse),
                        vp(ws), ws_bytes, None)


def test_invalid_arguments(lib):
    assert lib.fa_paged(None, *[vp(P)] * 11, 0, None) == 1
    for name in ("q", "kp", "v", "table", "lens", "cu", "o", "lse"):
        assert call(lib, **{name: 0}) == 1
    for kw in (dict(B=0), dict(T=0), dict(H=0), dict(H_kv=0), dict(max_q=0), dict(P=0), dict(max_pages=0), dict(T=-1),
               dict(H=3), dict(H=2, H_kv=4), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(causal=2), dict(quant=2), dict(window=-2), dict(window=8, causal=0),
               dict(quant=1), dict(quant=1, ks=P), dict(q_stride=(-256, 64)), dict(q_stride=(256, (1 << 31) + 8)),
               dict(max_pages=1 << 27, page=16), dict(P=1 << 30, H_kv=2), dict(T=1 << 30),
               dict(T=1 << 24, max_q=1 << 24, max_pages=1 << 22, H_kv=1, H=1)):   # more work than 32 bits count
        assert call(lib, **kw) == 1, kw


def test_unsupported_and_misaligned(lib):
    for kw in (dict(d=96), dict(d=256), dict(page=8), dict(page=48), dict(page=512), dict(dtype=2), dict(dtype=9),
               dict(H=258, H_kv=2)):
        assert call(lib, **kw) == 2, kw
    for kw in (dict(q=P + 8), dict(kp=P + 4), dict(v=P + 2), dict(o=P + 8), dict(lse=P + 2), dict(table=P + 2),
               dict(lens=P + 1), dict(cu=P + 3), dict(q_stride=(252, 64)), dict(q_stride=(256, 63)),
               dict(quant=1, ks=P + 8, vs=P)):
        assert call(lib, **kw) == 3, kw


@pytest.mark.skipif(not NO_GPU, reason="what a machine without a GPU answers")
def test_valid_calls_reach_the_device_check(lib):
    for kw in (dict(), dict(quant=1, ks=P, vs=P), dict(window=0), dict(causal=0), dict(max_q=1 << 20), dict(H=256, H_kv=2),
               # a prompt of 64K tokens, and 1024 sequences of up to a million keys
               dict(B=1, T=1 << 16, max_q=1 << 16, H=64, H_kv=8, P=1 << 14, max_pages=1 << 13),
               dict(B=1024, T=1024, max_q=1, H=32, H_kv=8, P=1 << 20, max_pages=1 << 16)):
        assert call(lib, **kw) == 4, kw
        assert lib.fa_paged_workspace_size(problem(**{k: v for k, v in kw.items() if k not in ("ks", "vs")})) == 0
    assert lib.fa_paged_workspace_size(None) == 0
