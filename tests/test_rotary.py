"""Rotary frequencies (host side): closed forms, limits of the scalings, refusals; and the
binding's refusals, which come before any device work."""
import contextlib
import itertools
import math
import random

import pytest
import torch

from exact_io_aware_93_b200 import api
from exact_io_aware_93_b200.rotary import rope_frequencies


def f(*a, **kw):
    return rope_frequencies(*a, device="cpu", **kw)


def test_plain_frequencies():
    freq, factor = f(64, base=10000.0)
    assert freq.dtype == torch.float64 and factor == 1.0
    for j in range(32):
        assert freq[j].item() == pytest.approx(10000.0 ** (-2.0 * j / 64), rel=1e-14)


def test_linear_divides_every_frequency():
    assert torch.equal(f(32, scaling="linear", scale=4.0)[0], f(32)[0] / 4.0)


def test_ntk_keeps_the_fastest_and_divides_the_slowest():
    plain, ntk = f(128)[0], f(128, scaling="ntk", scale=8.0)[0]
    assert ntk[0].item() == 1.0
    assert (plain[-1] / ntk[-1]).item() == pytest.approx(8.0, rel=1e-12)
    assert torch.all(ntk <= plain)


def test_bands_keep_fast_pairs_and_divide_slow_ones():
    plain = f(128, base=500000.0)[0]
    freq, factor = f(128, base=500000.0, scaling="bands", scale=8.0, trained=8192)
    turns = 8192 * plain / (2 * math.pi)
    assert factor == 1.0
    assert torch.equal(freq[turns >= 4.0], plain[turns >= 4.0])
    assert torch.allclose(freq[turns <= 1.0], plain[turns <= 1.0] / 8.0, rtol=1e-14)
    mid = (turns > 1.0) & (turns < 4.0)
    assert mid.any() and torch.all(freq[mid] < plain[mid]) and torch.all(freq[mid] > plain[mid] / 8.0)


def test_yarn_ends_and_factor():
    plain = f(128)[0]
    freq, factor = f(128, scaling="yarn", scale=16.0, trained=4096)
    assert factor == pytest.approx(0.1 * math.log(16.0) + 1.0)
    assert torch.equal(freq[:10], plain[:10])                   # more than 32 turns over 4096 positions
    assert torch.allclose(freq[-10:], plain[-10:] / 16.0, rtol=1e-14)
    assert torch.all(freq[1:] < freq[:-1])


@pytest.mark.parametrize("dim,base,scale,trained,low,high", [
    (128, 1e4, 16.0, 4096, 1.0, 32.0),                          # the slowest pair makes less than `low` turns
    (128, 1e4, 4.0, 65536, 1.0, 32.0), (64, 1e4, 4.0, 65536, 1.0, 32.0),
    (128, 1e4, 4.0, 131072, 1.0, 32.0), (64, 1e4, 4.0, 131072, 0.5, 64.0),   # and where it makes more
    (64, 100.0, 2.0, 65536, 1.0, 32.0), (2, 1e4, 2.0, 65536, 1.0, 32.0)])    # the end's limit, rotary_dim - 1
def test_yarn_blends_every_pair_by_the_definition(dim, base, scale, trained, low, high):
    """Pair x makes `turns` turns over `trained` positions where trained base^(-2x / dim) = 2 pi turns;
    the blend is linear in x from floor(x(high)) to ceil(x(low)), wherever the last pair is."""
    freq, _ = f(dim, base=base, scaling="yarn", scale=scale, trained=trained, low=low, high=high)

    def at(turns):
        return dim / 2 * math.log(trained / (2 * math.pi * turns)) / math.log(base)
    first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), dim - 1)
    for x in range(dim // 2):
        part = min(max((x - first) / (last - first), 0.0), 1.0) if last > first else float(x > first)
        plain = base ** (-2.0 * x / dim)
        want = plain * (1.0 - part) + plain / scale * part
        assert freq[x].item() == pytest.approx(want, rel=1e-12), x


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, scale=0.5),
    dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, scaling="yarn", scale=2.0),
    dict(rotary_dim=64, scaling="bands", scale=2.0, trained=100, low=4.0, high=1.0),
    dict(rotary_dim=2, scaling="ntk", scale=2.0),
])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        f(**kw)


def test_binding_refuses_before_device_work():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.arange(4), f(64)[0]
    with pytest.raises(ValueError):
        api.rope(q, None, pos, freq)                            # no CPU path
    with pytest.raises(TypeError):
        api.rope(q.float(), None, pos, freq)
    with pytest.raises(ValueError):
        api.rope(q[0], None, pos, freq)                         # two dimensions
    with pytest.raises(ValueError):
        api.cache_append(q, q, q, q, pos, pos, pos)


@pytest.mark.parametrize("make", [
    lambda x: x.expand(3, 4, 2, 64)[:, :, :, :],                # a batch stride of 0
    lambda x: torch.as_strided(x, (3, 4, 2, 64), (512, 128, 32, 1)),   # heads overlap
])
def test_rope_outputs_may_not_overlap_themselves(make, monkeypatch):
    monkeypatch.setattr(api, "_check_heads", lambda *a: None)
    x = torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlap itself"):
        api._check_rope_out("q_out", make(torch.zeros(4096, dtype=torch.bfloat16)[:512].view(1, 4, 2, 64)), x)


def test_rope_output_apart_from_its_inputs(monkeypatch):
    monkeypatch.setattr(api, "_check_heads", lambda *a: None)
    buf = torch.zeros(10, 6, 64, dtype=torch.bfloat16)
    q, k = buf[:8, :4], buf[:8, 4:]
    api._check_rope_out("q_out", q, q, k)                       # in place, beside k
    api._check_rope_out("q_out", torch.zeros(8, 4, 64, dtype=torch.bfloat16), q, k)
    with pytest.raises(ValueError):
        api._check_rope_out("q_out", buf[1:9, :4], q, k)        # shifted by a token
    with pytest.raises(ValueError):
        api._check_rope_out("k_out", q, q[:, :4], q)            # another input too


def test_buffers_that_overlap():
    buf = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    k, v = buf[:2], buf[2:]
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    api._check_pools(k, v, rows, rows)                          # two halves of one pool
    for a, b, r in ((k, k, rows), (buf[:3], buf[1:], rows), (k, v, v[0, 0, :3])):
        with pytest.raises(ValueError):
            api._check_pools(a, b, r)
    api._check_apart("out", k, v, None, rows, rows[:0])
    with pytest.raises(ValueError):
        api._check_apart("out", k, rows, buf[1:3])


class _Reached(Exception):
    """The library would have been called."""


def _no_device(monkeypatch):
    """The binding's checks on CPU tensors: only where a tensor lies is overlooked."""
    def reached():
        raise _Reached
    monkeypatch.setattr(api, "_check_heads", lambda *a: None)
    monkeypatch.setattr(api, "_on", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_stream_ptr", lambda t: 0)
    monkeypatch.setattr(api, "lib", reached)


def _rotate(q, k, q_out=None, k_out=None):
    api.rope(q, k, torch.arange(q.shape[-3]), f(64)[0], q_out=q_out, k_out=k_out)


def test_rope_outputs_that_overlap_each_other_or_an_input(monkeypatch):
    _no_device(monkeypatch)
    x = torch.zeros(8, 8, 64, dtype=torch.bfloat16)
    fused, other = x.clone(), torch.zeros(8, 8, 64, dtype=torch.bfloat16)
    q, k = fused[:, :4], fused[:, 4:8]
    heads = torch.zeros(2, 6, 8, 64, dtype=torch.bfloat16).transpose(1, 2)          # [B, N, H, d] of [B, H, N, d]
    for q_, k_, qo, ko in (
            (q, k, q, k), (q, k, None, None), (q, k, q, None), (q, k, None, k),    # in place, whole or in part
            (q, k, other[:, :4], other[:, 4:]), (q, k, other[:, 4:], other[:, :4]), (q, k, other[:, :4], k),
            (x[:4], x[4:], x[:4], x[4:]), (x[:1, :3], x[:1, 3:6], x[:1, :3], x[:1, 3:6]),
            (heads[:, :, :4], heads[:, :, 4:], heads[:, :, :4], heads[:, :, 4:]),
            (x.view(2, 4, 8, 64)[:, :, :5], x.view(2, 4, 8, 64)[:, :, 5:], x.view(2, 4, 8, 64)[:, :, :5], None),
            (x[:, 1:1], x[:, :2], None, x[:, :2]), (x[:, :2], x[:, 1:1], x[:, :2], x[:, 1:1]), (q, None, q, None)):
        with pytest.raises(_Reached):
            _rotate(q_, k_, qo, ko)
    for q_, k_, qo, ko in (
            (q, k, other[:, :4], other[:, :4]),                                     # one buffer for both
            (q, k, other[:, :4], other[:, 2:6]), (q, k, q, q), (q, k, k, None),
            (x[:, :4], x[:, 2:6], x[:, :4], x[:, 2:6]),                             # inputs that share heads, in place
            (x[:, :4], x[:, 2:6], x[:, :4], None), (x[:, :4], x[:, 2:6], None, x[:, 2:6]),
            (x[:, :4], x[:, 3:], x[:, :4], other[:, 3:]),
            (x[:4, :4], x[3:7, :4], x[:4, :4], other[:4, :4]),                      # or a token
            (heads[:, :, :4], heads[:, :, 3:6], heads[:, :, :4], None)):
        with pytest.raises(ValueError):
            _rotate(q_, k_, qo, ko)


def test_interleaved_slices_have_no_element_in_common():
    """Whatever the strides: where slices are taken for interleaved, no offset is in both."""
    rng = random.Random(7)
    buf, found = torch.zeros(4096, dtype=torch.bfloat16), 0
    strides = [0, 1, 2, 3, 4, 6, 8, 12, 24, 48, 96, 7]
    for _ in range(20000):
        pair = []
        for _ in range(2):
            shape = [rng.randint(1, 4) for _ in range(3)] + [rng.randint(1, 6)]
            pair.append(torch.as_strided(buf, shape, [rng.choice(strides) for _ in range(3)] + [1], rng.randint(0, 120)))
        if api._interleaved(*pair):
            found += 1
            at = [{t.storage_offset() + sum(i * s for i, s in zip(ix, t.stride()))
                   for ix in itertools.product(*map(range, t.shape))} for t in pair]
            assert not at[0] & at[1], [(t.shape, t.stride(), t.storage_offset()) for t in pair]
    assert found > 500


def test_new_rows_that_run_into_a_pool():
    flat = torch.zeros(8192, dtype=torch.bfloat16)
    a, b = flat[2048:4096].view(2, 1, 16, 64), flat[6144:].view(2, 1, 16, 64)
    for first, t, apart in ((0, 16, True), (0, 17, False), (1920, 1, True), (1984, 1, False), (2048, 1, False),
                            (3968, 1, False), (4032, 1, True), (4096, 16, True), (4096, 17, False)):
        rows = torch.as_strided(flat, (t, 1, 64), (128, 64, 1), first + 64)     # the second half of each 128
        if apart:
            api._check_pools(a, b, flat[:64].view(1, 1, 64), rows)
        else:
            with pytest.raises(ValueError):
                api._check_pools(a, b, flat[:64].view(1, 1, 64), rows)
            with pytest.raises(ValueError):
                api._check_pools(b, a, rows)
    api._check_pools(a, b, flat[2112:2112].view(0, 1, 64))
