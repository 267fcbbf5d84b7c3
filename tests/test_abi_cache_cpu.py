"""Refusals of the rotary and paged-cache entry points: documented codes, before any device work."""
import ctypes

import pytest
import torch

from exact_io_aware_93_b200 import build as fabuild
from exact_io_aware_93_b200.api import FaCacheProblem, FaRopeProblem

P = 0x10000
OK_HERE = 0 if torch.cuda.is_available() else 4     # a valid call gets as far as the device check
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(fabuild.build())
    L.fa_rope.argtypes = [ctypes.POINTER(FaRopeProblem)] + [vp] * 7
    L.fa_cache_append.argtypes = [ctypes.POINTER(FaCacheProblem)] + [vp] * 10
    L.fa_cache_gather.argtypes = [ctypes.POINTER(FaCacheProblem)] + [vp] * 11
    return L


def test_rope_codes(lib):
    def call(q=P, k=P, qo=P, ko=P, pos=P, freq=P, **kw):
        base = dict(B=1, N=4, H=2, H_k=1, d=64, rotary_dim=64, interleaved=0, inverse=0, factor=1.0, dtype=0, pos64=0,
                    q_stride=(0, 128, 64), k_stride=(0, 64, 64), q_out_stride=(0, 128, 64), k_out_stride=(0, 64, 64),
                    pos_stride=(0, 1))
        base.update(kw)
        p = FaRopeProblem(**base)
        return lib.fa_rope(ctypes.byref(p), vp(q), vp(k), vp(qo), vp(ko), vp(pos), vp(freq), None)
    assert lib.fa_rope(None, vp(P), vp(P), vp(P), vp(P), vp(P), vp(P), None) == 1
    assert call(q=0) == 1 and call(qo=0) == 1 and call(pos=0) == 1 and call(freq=0) == 1
    assert call(k=0) == 1 and call(ko=0) == 1            # H_k = 1 without k
    assert call(H_k=0) == 1                              # k without heads
    assert call(B=0) == 1 and call(N=0) == 1 and call(H=0) == 1 and call(H_k=-1) == 1
    assert call(rotary_dim=63) == 1 and call(rotary_dim=66) == 1 and call(rotary_dim=0) == 1
    assert call(d=1) == 1 and call(d=2048, rotary_dim=64) == 1
    assert call(interleaved=2) == 1 and call(inverse=-1) == 1 and call(pos64=2) == 1
    assert call(factor=float("nan")) == 1 and call(factor=float("inf")) == 1
    assert call(dtype=2) == 2 and call(dtype=7) == 2
    assert call(q=P + 1) == 3 and call(pos=P + 2) == 3 and call(freq=P + 4) == 3
    assert call(pos=P + 4, pos64=1) == 3
    if OK_HERE == 4:
        assert call() == 4 and call(q=P + 2) == 4 and call(k=0, ko=0, H_k=0) == 4


def cache(**kw):
    base = dict(B=2, T=5, H_kv=2, d=64, P=9, max_pages=4, page=16, dtype=0, quant=0, k_stride=(128, 64),
                v_stride=(128, 64))
    base.update(kw)
    return ctypes.byref(FaCacheProblem(**base))


def test_cache_append_codes(lib):
    def call(k=P, v=P, kp=P, vpg=P, ks=0, vs=0, table=P, lens=P, cu=P, **kw):
        return lib.fa_cache_append(cache(**kw), vp(k), vp(v), vp(kp), vp(vpg), vp(ks), vp(vs), vp(table), vp(lens),
                                   vp(cu), None)
    assert lib.fa_cache_append(None, *[vp(P)] * 9, None) == 1
    for name in ("k", "v", "kp", "vpg", "table", "lens", "cu"):
        assert call(**{name: 0}) == 1
    assert call(B=0) == 1 and call(T=0) == 1 and call(H_kv=0) == 1 and call(P=0) == 1 and call(max_pages=0) == 1
    assert call(quant=2) == 1 and call(quant=1) == 1      # e4m3 pages need scales
    assert call(d=96) == 2 and call(page=8) == 2 and call(page=48) == 2 and call(page=512) == 2 and call(dtype=2) == 2
    assert call(k=P + 8) == 3 and call(vpg=P + 4) == 3 and call(cu=P + 2) == 3
    assert call(k_stride=(124, 64)) == 3
    if OK_HERE == 4:
        assert call() == 4 and call(quant=1, ks=P + 1, vs=P) == 4


def test_cache_gather_codes(lib):
    def call(kp=P, vpg=P, ks=0, vs=0, table=P, lens=P, cu=P, starts=0, ko=P, vo=P, **kw):
        return lib.fa_cache_gather(cache(**kw), vp(kp), vp(vpg), vp(ks), vp(vs), vp(table), vp(lens), vp(cu),
                                   vp(starts), vp(ko), vp(vo), None)
    assert lib.fa_cache_gather(None, *[vp(P)] * 10, None) == 1
    for name in ("kp", "vpg", "table", "lens", "cu", "ko", "vo"):
        assert call(**{name: 0}) == 1
    assert call(quant=1, ks=P) == 1 and call(T=-1) == 1
    assert call(d=256) == 2 and call(page=100) == 2
    assert call(ko=P + 8) == 3 and call(starts=P + 1) == 3
    if OK_HERE == 4:
        assert call() == 4 and call(quant=1, ks=P, vs=P, starts=P) == 4
