"""Rotary positions, the paged cache and attention over it through the checking build: every TMA
coordinate and global index compared with its tensor's extent.  No check may fire, and the results
are the release build's bit for bit."""
import pytest
import torch

from exact_io_aware_93_b200 import api
from tests import test_cache_gpu, test_paged_gpu
from tests.paged import offsets

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture
def both(monkeypatch):
    """Runs a call with the release library and with the checking build: the two results."""
    def run(call):
        want = call()
        torch.cuda.synchronize()
        assert api.get_status_site() == (0, 0)
        with monkeypatch.context() as m:
            m.setenv("FA_B200_CHECKS", "1")
            m.setattr(api, "_lib", None)
            assert api.lib().fa_checks_enabled() == 1
            got = call()
            torch.cuda.synchronize()
            assert api.get_status_site() == (0, 0)
        return want, got
    return run


def same(want, got):
    assert len(want) == len(got)
    for x, y in zip(want, got):
        assert torch.equal(test_cache_gpu.bits(x), test_cache_gpu.bits(y))


@pytest.mark.parametrize("t,h,hk,d,rd,dtype,inter", [(1, 1, 1, 64, 64, BF, False), (777, 5, 3, 128, 64, FP, True),
                                                     (3000, 3, 1, 40, 30, BF, False), (65, 32, 8, 128, 128, BF, True)])
def test_rotation_passes_every_check(both, t, h, hk, d, rd, dtype, inter):
    x = torch.randn(t, h + hk, d, device="cuda").to(dtype)
    freq = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64, device="cuda") * 2 / rd)
    pos = torch.arange(t, device="cuda")
    same(*both(lambda: api.rope(x[:, :h], x[:, h:], pos, freq, interleaved=inter)
               + api.rope_bwd(x[:, :h], x[:, h:], pos, freq, interleaved=inter)))


@pytest.mark.parametrize("new,lens,hk,d,page,dtype,quant", [
    ([1, 0, 33], [1, 5, 700], 3, 64, 16, BF, True), ([500, 1], [500, 300], 2, 128, 256, FP, False),
    ([1] * 40, [13 * i + 1 for i in range(40)], 1, 64, 32, FP, True), ([5000], [6000], 1, 64, 128, BF, True)])
def test_cache_passes_every_check(both, new, lens, hk, d, page, dtype, quant):
    def call():
        s = test_cache_gpu.build(new, lens, hk, d, page, dtype, quant, seed=31)
        test_cache_gpu.append(s)
        out = [torch.zeros(sum(lens) + 3, hk, d, dtype=dtype, device="cuda") for _ in "kv"]
        api.cache_gather(*s["pages"], s["table"], s["seqlens"], offsets(new).cuda(), sum(new),
                         starts=s["seqlens"] - torch.tensor(new, dtype=torch.int32, device="cuda"),
                         k_scales=s["scales"][0], v_scales=s["scales"][1], dtype=dtype, k_out=out[0][:sum(new)],
                         v_out=out[1][:sum(new)])
        return s["pages"] + [x for x in s["scales"] if x is not None] + out
    same(*both(call))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens,h,hk,d,page,causal,window", [
    ([1] * 5, [130, 1, 129, 2000, 77], 8, 2, 128, 64, True, -1),
    ([3, 2, 0], [700, 2, 9], 4, 4, 64, 256, True, 100),
    ([200, 333], [200, 1000], 4, 2, 128, 32, True, -1),
    ([90, 1, 1], [300, 1500, 40], 6, 2, 64, 16, False, -1),
    ([260, 3], [1030, 700], 5, 1, 128, 128, True, 300),
])
def test_paged_attention_passes_every_check(both, new, lens, h, hk, d, page, causal, window, dtype, quant):
    s = test_paged_gpu.build(new, lens, h, hk, d, page, dtype, quant, seed=32, window=window)
    same(*both(lambda: test_paged_gpu.attend(s, causal)))
