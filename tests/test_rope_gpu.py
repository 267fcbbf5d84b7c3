"""Rotary positions and their gradient through fa_rope, against the rotation in fp64.

Tolerance: the output's rounding, half a step (eps / 2 of the value; half of the smallest
subnormal below that), plus the fp32 work: the reduced angle is rounded to 32 bits (at most
2^-26 turns = 2^-23 rad), sine and cosine are good to 2 units and the two products and their
sum round once each, all together below factor * (|a| + |b|) * 2^-21."""
import pytest
import torch

from exact_io_aware_93_b200 import api
from exact_io_aware_93_b200.rotary import rope_frequencies

pytestmark = pytest.mark.gpu


def reference(x, positions, inv_freq, interleaved, factor, inverse=False):
    """(value, tolerance) in fp64 on the CPU."""
    x64, pos, freq = x.double().cpu(), positions.cpu().double(), inv_freq.cpu()
    half = freq.numel()
    ang = (pos[..., None] * freq)[..., None, :] * (-1.0 if inverse else 1.0)
    c, s = torch.cos(ang) * factor, torch.sin(ang) * factor
    i = torch.arange(half)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, slack = x64.clone(), torch.zeros_like(x64)
    a, b = x64[..., i0], x64[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    slack[..., i0] = slack[..., i1] = abs(factor) * (a.abs() + b.abs()) * 2.0 ** -21
    step = torch.finfo(x.dtype)
    return y, step.eps / 2 * (y.abs() + slack) + step.smallest_normal * step.eps / 2 + slack


def check(got, x, positions, inv_freq, interleaved, factor, inverse=False):
    want, tol = reference(x, positions, inv_freq, interleaved, factor, inverse)
    err = (got.double().cpu() - want).abs()
    assert torch.all(err <= tol), (err - tol).max()


CASES = [
    # shape (tokens or batch x tokens), heads, kv heads, d, rotary, dtype, interleaved, factor, first position
    ((1,), 1, 1, 64, 64, torch.bfloat16, False, 1.0, 0),
    ((1,), 3, 0, 128, 128, torch.float16, True, 1.0, 131071),
    ((16,), 32, 8, 128, 128, torch.bfloat16, False, 1.0, 30000),
    ((7,), 5, 1, 64, 32, torch.bfloat16, True, 1.25, 2 ** 31 - 8),      # far positions
    ((3001,), 4, 2, 128, 64, torch.float16, False, 1.139, 100),
    ((129,), 3, 2, 64, 54, torch.bfloat16, False, 1.0, 77),             # rotary not a multiple of 16
    ((65,), 2, 2, 64, 2, torch.float16, True, 0.5, 5),
    ((50,), 2, 1, 80, 80, torch.bfloat16, False, 1.0, 9),               # other head sizes
    ((50,), 2, 1, 75, 46, torch.float16, True, 1.0, 9),                 # odd head size
    ((2, 300), 6, 2, 128, 128, torch.bfloat16, False, 1.0, 0),
    ((3, 1200), 16, 16, 128, 96, torch.bfloat16, True, 1.0, 8000),
    ((20,), 1, 1, 1024, 1024, torch.bfloat16, False, 1.0, 3),
    ((20003,), 1, 0, 64, 32, torch.float16, False, 1.0, 11),            # 16 tokens to a block
    ((9000, 1), 3, 1, 64, 64, torch.bfloat16, True, 1.0, 5),            # one token per batch row
    ((1700, 7), 5, 0, 128, 64, torch.float16, False, 1.0, 0),
    ((5000, 3), 2, 1, 75, 46, torch.bfloat16, False, 1.0, 4),
]


@pytest.mark.parametrize("lead,h,hk,d,rd,dtype,inter,factor,first", CASES)
def test_rope_and_its_gradient(lead, h, hk, d, rd, dtype, inter, factor, first):
    g = torch.Generator().manual_seed(h * 1000 + d + rd)
    q = torch.randn(*lead, h, d, generator=g).to(dtype).cuda()
    k = torch.randn(*lead, hk, d, generator=g).to(dtype).cuda() if hk else None
    freq, _ = rope_frequencies(rd)
    pos = first + torch.arange(lead[-1], device="cuda")
    for p in (pos, pos.to(torch.int32)):
        for fn, inverse in ((api.rope, False), (api.rope_bwd, True)):
            yq, yk = fn(q, k, p, freq, interleaved=inter, factor=factor)
            check(yq, q, pos, freq, inter, factor, inverse)
            if hk:
                check(yk, k, pos, freq, inter, factor, inverse)
            else:
                assert yk is None


@pytest.mark.parametrize("inter", [False, True])
def test_rope_strided_slices_in_place_and_per_row_positions(inter):
    """Slices of a fused projection, rotated in place: the values between them keep their bits;
    positions differ per batch row, run backwards and may be negative."""
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(2, 200, 10, 64, generator=g).to(torch.bfloat16).cuda()
    before = qkv.clone()
    pos = torch.randint(-5000, 5000, (2, 200), generator=g).cuda().flip(1)
    freq, _ = rope_frequencies(64)
    q, k = qkv[:, :, :6], qkv[:, :, 6:8]
    yq, yk = api.rope(q, k, pos, freq, interleaved=inter, q_out=q, k_out=k)
    assert yq is q and yk is k
    check(q, before[:, :, :6], pos, freq, inter, 1.0)
    check(k, before[:, :, 6:8], pos, freq, inter, 1.0)
    assert torch.equal(qkv[:, :, 8:], before[:, :, 8:])
    # a buffer with rows that are not 16-byte aligned gives the same bits
    wide = torch.zeros(2, 200, 6, 67, dtype=torch.bfloat16, device="cuda")
    out = wide[..., 1:65]
    api.rope(before[:, :, :6], None, pos, freq, interleaved=inter, q_out=out)
    assert torch.equal(out, q) and torch.all(wide[..., 0] == 0) and torch.all(wide[..., 65:] == 0)


def test_rope_of_broadcast_positions_and_batches():
    freq, _ = rope_frequencies(128)
    q = torch.randn(3, 50, 2, 128, device="cuda").to(torch.float16)
    pos = torch.arange(50, device="cuda")
    a, _ = api.rope(q, None, pos, freq)
    b, _ = api.rope(q, None, pos.expand(3, 50), freq)
    c, _ = api.rope(q.view(150, 2, 128), None, pos.repeat(3), freq)
    assert torch.equal(a, b) and torch.equal(a.view(150, 2, 128), c)
    one = q[:1].expand(3, 50, 2, 128)                       # the same queries for three batch rows
    d, _ = api.rope(one, None, pos, freq)
    assert torch.equal(d[0], d[2]) and torch.equal(d[0], a[0])


def test_rope_gradient_against_differences():
    """The gradient of L = sum(w o rope(x)) along a direction u equals the difference quotient of
    the (linear) fp64 rotation, computed from rope's own gradient in fp64 sums."""
    g = torch.Generator().manual_seed(9)
    x, u, w = (torch.randn(40, 3, 64, generator=g).to(torch.float16) for _ in range(3))
    freq, factor = rope_frequencies(48, scaling="yarn", scale=4.0, trained=4096)
    pos = torch.arange(40) * 997
    grad, _ = api.rope_bwd(w.cuda(), None, pos.cuda(), freq, factor=factor)
    h = 0.5
    up, down = (_rotated64(x.double() + e * u.double(), pos, freq.cpu(), factor) for e in (h, -h))
    quotient = ((up - down) * w.double()).sum() / (2 * h)
    got = (grad.double().cpu() * u.double()).sum()
    # the gradient's elements round to fp16: eps / 2 each, at most the sum of |grad u| eps
    tol = (grad.double().cpu() * u.double()).abs().sum() * torch.finfo(torch.float16).eps
    assert abs(got - quotient) <= tol, (got, quotient, tol)


def _rotated64(v, pos, freq, factor):
    half = freq.numel()
    ang = (pos.double()[:, None] * freq)[:, None, :]
    a, b = v[..., :half], v[..., half:2 * half]
    c, s = torch.cos(ang) * factor, torch.sin(ang) * factor
    return torch.cat((a * c - b * s, b * c + a * s, v[..., 2 * half:]), -1)


def test_rope_non_finite_values_stay_in_their_pair():
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 0, 3] = float("nan")
    x[2, 1, 5] = float("inf")
    freq, _ = rope_frequencies(64)
    y, _ = api.rope(x, None, torch.arange(4, device="cuda"), freq)
    bad = ~torch.isfinite(y)
    where = {tuple(i) for i in bad.nonzero().tolist()}
    assert where <= {(1, 0, 3), (1, 0, 35), (2, 1, 5), (2, 1, 37)} and (1, 0, 3) in where and (2, 1, 5) in where


def test_rope_captured_replayed_and_on_another_stream():
    freq, _ = rope_frequencies(128)
    q = torch.randn(33, 4, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(33, device="cuda", dtype=torch.int32)
    want, _ = api.rope(q, None, pos + 50, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = api.rope(q, None, pos + 50, freq)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rope(q, None, pos, freq, q_out=out)
    pos += 50
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert api.get_status() == 0


def test_rope_empty_and_refused():
    freq, _ = rope_frequencies(64)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(4, device="cuda")
    y, _ = api.rope(q[:0], None, pos[:0], freq)
    assert y.shape == (0, 2, 64)
    for bad in (dict(positions=pos[:3]), dict(positions=pos.float()), dict(positions=pos.cpu()),
                dict(inv_freq=freq.float()), dict(inv_freq=torch.ones(33, dtype=torch.float64, device="cuda")),
                dict(k=q[:3]), dict(k=q.half()), dict(k_out=q)):
        kw = {"k": None, "positions": pos, "inv_freq": freq, **bad}
        with pytest.raises((ValueError, TypeError)):
            api.rope(q, kw.pop("k"), kw.pop("positions"), kw.pop("inv_freq"), **kw)
    with pytest.raises(api.FAError):
        api.rope(q, None, pos, freq, factor=float("inf"))
