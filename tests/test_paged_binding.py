"""The paged calls' checks of the caller's buffers, on CPU tensors: no device work comes before them."""
import contextlib

import pytest
import torch

from exact_io_aware_93_b200 import api

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


class _Reached(Exception):
    """The library would have been called."""


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    def reached():
        raise _Reached
    monkeypatch.setattr(api, "_check_heads", lambda *a: None)
    monkeypatch.setattr(api, "_check_pages", lambda k, v, t, s, ks, vs, dtype: ks is not None)
    monkeypatch.setattr(api, "_on", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_stream_ptr", lambda t: 0)
    monkeypatch.setattr(api, "lib", reached)


POOL, SCALES = ((4, 2, 16, 64), BF), ((4, 2, 16), U8)
READ = dict(k_pages=POOL, v_pages=POOL, page_table=((2, 4), I32), seqlens=((2,), I32), k_scales=SCALES, v_scales=SCALES)
PAGED = dict(READ, q=((3, 4, 64), BF), cu_q=((3,), I32))
PAGED_WRITTEN = dict(out=((3, 4, 64), BF), lse=((4, 3), torch.float32), workspace=((4096,), U8))
GATHER = dict(READ, cu_k=((3,), I32), starts=((2,), I32))
GATHER_WRITTEN = dict(k_out=((5, 2, 64), BF), v_out=((5, 2, 64), BF))


def tensors(kinds):
    return {name: torch.zeros(shape, dtype=dtype) for name, (shape, dtype) in kinds.items()}


def sharing(first, second, at):
    """Tensors of these kinds in one buffer: the second begins `at` bytes in."""
    size = [torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size() for shape, dtype in (first, second)]
    buf = torch.zeros(size[0] + size[1] + 8, dtype=U8)
    return [buf[lo:lo + n].view(dtype).view(shape) for lo, n, (shape, dtype) in ((0, size[0], first), (at, size[1], second))]


@pytest.mark.parametrize("call,read,written,more", [
    (api.paged_attention, PAGED, PAGED_WRITTEN, dict(max_q=2)), (api.cache_gather, GATHER, GATHER_WRITTEN, dict(total=5))])
def test_given_buffers_lie_apart_from_what_is_read_and_from_each_other(call, read, written, more):
    with pytest.raises(_Reached):
        call(**tensors(read), **tensors(written), **more)
    every = {**read, **written}
    for name, kind in written.items():
        for other in every:
            if other == name:
                continue
            end = torch.Size(every[other][0]).numel() * torch.empty(0, dtype=every[other][1]).element_size()
            for at in (0, end - 8):                              # from its beginning, over its last bytes
                t, w = sharing(every[other], kind, at)
                args = {**tensors(read), **tensors(written), other: t, name: w}
                with pytest.raises(ValueError, match="overlap"):
                    call(**args, **more)
            t, w = sharing(every[other], kind, (end + 7) // 8 * 8)
            with pytest.raises(_Reached):
                call(**{**tensors(read), **tensors(written), other: t, name: w}, **more)
