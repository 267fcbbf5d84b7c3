"""The operators around attention together, as a model's step calls them: rotary positions on
slices of a fused projection, the new keys and values into a paged cache, attention against it
(prompt chunks, mixed batches, single tokens, drafted tokens and their rejection); and in training
rotary positions, attention, its backward pass and the rotation's."""
import pytest
import torch

from exact_io_aware_93_b200 import api
from exact_io_aware_93_b200.rotary import rope_frequencies
from tests.paged import offsets, page_tables, quantise_rows
from tests.parity import GRAD_TOL
from tests.test_paged_gpu import check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

# new tokens of the three sequences; a negative number takes back that many (rejected drafts)
STEPS = [(100, 0, 0), (60, 1, 0), (1, 130, 7), (1, 1, 1), (4, 4, 4), (-2, -3, 0), (1, 1, 1), (3, 0, 2), (1, 1, 1)]


@pytest.mark.parametrize("dtype,quant,d,page,window", [(BF, False, 128, 16, -1), (BF, True, 128, 64, -1),
                                                       (FP, True, 64, 32, 50), (FP, False, 64, 128, -1)])
def test_steps_of_a_served_batch(dtype, quant, d, page, window):
    h, hk, total = 8, 2, 320
    g = torch.Generator().manual_seed(21)
    table, pool = page_tables([total] * 3, page, g)
    table = table.cuda()
    shape = (pool, hk, page, d)
    if quant:
        pages = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv"]
        scales = [torch.zeros(shape[:3], dtype=torch.float8_e8m0fnu, device="cuda") for _ in "kv"]
    else:
        pages = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in "kv"]
        scales = [None, None]
    freq, factor = rope_frequencies(d, scaling="yarn", scale=8.0, trained=64)
    lens = [0, 0, 0]
    held = [[torch.zeros(0, hk, d, dtype=torch.float64) for _ in range(3)] for _ in "kv"]   # as the cache holds them
    for step in STEPS:
        if min(step) < 0:
            lens = [m + n for m, n in zip(lens, step)]
            for vals in held:
                for b in range(3):
                    vals[b] = vals[b][:lens[b]]
            continue
        new, T = list(step), sum(step)
        lens = [m + n for m, n in zip(lens, new)]
        qkv = torch.randn(T, h + 2 * hk, d, generator=g).to(dtype).cuda()
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        pos = torch.cat([torch.arange(m - n, m) for n, m in zip(new, lens)]).to(torch.int32).cuda()
        api.rope(q, k, pos, freq, factor=factor, q_out=q, k_out=k)
        seqlens, cu = torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets(new).cuda()
        api.cache_append(k, v, *pages, table, seqlens, cu, k_scales=scales[0], v_scales=scales[1])
        o, lse = api.paged_attention(q, *pages, table, seqlens, cu, max(new), window=None if window < 0 else window,
                                     k_scales=scales[0], v_scales=scales[1])
        torch.cuda.synchronize()
        assert api.get_status_site() == (0, 0)
        for vals, x in zip(held, (k, v)):
            rows = quantise_rows(x)[0] if quant else x.double().cpu()
            for b in range(3):
                vals[b] = torch.cat([vals[b], rows[cu[b]:cu[b + 1]]])
        s = dict(new=new, lens=lens, window=window, h=h, hk=hk, values=held, scales=scales, q=q)
        check(s, o, lse)
    cu = offsets(lens).cuda()
    back = api.cache_gather(*pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, sum(lens),
                            k_scales=scales[0], v_scales=scales[1], dtype=dtype)
    for x, vals in zip(back, held):
        assert torch.equal(x.double().cpu(), torch.cat(vals))


def test_chunks_of_a_prompt_give_what_the_whole_prompt_gives():
    """A prompt in chunks against its cache, and the forward pass over all of it: both within the
    fp64 check's bounds."""
    n, h, hk, d, page = 700, 8, 2, 128, 32
    g = torch.Generator().manual_seed(22)
    table, pool = page_tables([n], page, g)
    table = table.cuda()
    pages = [torch.full((pool, hk, page, d), float("nan"), dtype=BF, device="cuda") for _ in "kv"]
    q, k, v = (torch.randn(n, x, d, generator=g).to(BF).cuda() for x in (h, hk, hk))
    s = dict(new=[n], lens=[n], window=-1, h=h, hk=hk, values=[[k.double().cpu()], [v.double().cpu()]],
             scales=[None, None], q=q)
    o, lse = api.fwd(q[None], k[None], v[None], causal=True)
    check(s, o[0], lse[0])
    o, lse = torch.zeros_like(q), torch.zeros(h, n, device="cuda")
    at = 0
    for m in (1, 255, 129, 315):
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        seqlens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
        api.cache_append(k[at:at + m], v[at:at + m], *pages, table, seqlens, cu)
        o[at:at + m], lse[:, at:at + m] = api.paged_attention(q[at:at + m], *pages, table, seqlens, cu, m)
        at += m
    assert at == n and api.get_status() == 0
    check(s, o, lse)


def test_rotation_in_a_training_step():
    """Gradients of the fused projection through rope, fwd, bwd and rope_bwd, against fp64 autograd."""
    b, n, h, hk, d = 2, 300, 4, 2, 64
    g = torch.Generator().manual_seed(23)
    qkv = torch.randn(b, n, h + 2 * hk, d, generator=g).to(BF)
    do = torch.randn(b, n, h, d, generator=g).to(BF)
    freq, factor = rope_frequencies(d)
    pos = torch.arange(n, device="cuda")
    x = qkv.cuda()
    q, k = api.rope(x[:, :, :h], x[:, :, h:h + hk], pos, freq)
    v = x[:, :, h + hk:].contiguous()
    o, lse = api.fwd(q, k, v, causal=True)
    dq, dk, dv = api.bwd(q, k, v, o, do.cuda(), lse, causal=True)
    dx = torch.zeros_like(x)
    api.rope_bwd(dq, dk, pos, freq, q_grad=dx[:, :, :h], k_grad=dx[:, :, h:h + hk])
    dx[:, :, h + hk:] = dv
    torch.cuda.synchronize()
    assert api.get_status() == 0

    y = qkv.double().requires_grad_()
    ang = torch.arange(n, dtype=torch.float64)[:, None] * freq.cpu()
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def turn(t):
        a, e = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([a * c - e * s, e * c + a * s], -1)
    qq, kk, vv = (t.transpose(1, 2) for t in (turn(y[:, :, :h]), turn(y[:, :, h:h + hk]), y[:, :, h + hk:]))
    kk, vv = (t.repeat_interleave(h // hk, 1) for t in (kk, vv))
    w = (qq @ kk.transpose(2, 3)) * d ** -0.5
    w = w.masked_fill(torch.ones(n, n).triu(1).bool(), float("-inf")).softmax(-1)
    (w @ vv).transpose(1, 2).backward(do.double())
    for part in (slice(0, h), slice(h, h + hk), slice(h + hk, h + 2 * hk)):
        want, got = y.grad[:, :, part], dx[:, :, part].double().cpu()
        assert ((got - want).abs().max() / want.abs().max()).item() <= GRAD_TOL
