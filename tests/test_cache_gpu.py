"""The paged key/value cache through fa_cache_append and fa_cache_gather: 16-bit pages move
bits; e4m3 pages hold exactly the definition's codes (power-of-two scales make every step
exact, so no tolerance is needed)."""
import pytest
import torch

from exact_io_aware_93_b200 import api
from tests.paged import locate, offsets, page_tables, quantise_rows

pytestmark = pytest.mark.gpu


def build(new, lens, hk, d, page, dtype, quant, seed, spread=1.0):
    """A cache of stale NaN with `new` rows to append; everything on the GPU."""
    g = torch.Generator().manual_seed(seed)
    table, pool = page_tables(lens, page, g)
    T = sum(new)
    qkv = (torch.randn(T, 3 * hk, d, generator=g) * torch.exp(spread * torch.randn(T, 3 * hk, 1, generator=g))).to(dtype)
    s = dict(table=table.cuda(), seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=offsets(new).cuda(),
             qkv=qkv.cuda())
    s["k"], s["v"] = s["qkv"][:, hk:2 * hk], s["qkv"][:, 2 * hk:]
    shape = (pool, hk, page, d)
    if quant:
        s["pages"] = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
        s["scales"] = [torch.full(shape[:3], 131, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in "kv"]
    else:
        s["pages"] = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in "kv"]
        s["scales"] = [None, None]
    return s


def append(s, **kw):
    a = dict(k=s["k"], v=s["v"], k_pages=s["pages"][0], v_pages=s["pages"][1], page_table=s["table"],
             seqlens=s["seqlens"], cu_q=s["cu"], k_scales=s["scales"][0], v_scales=s["scales"][1])
    a.update(kw)
    api.cache_append(**a)


def bits(t):
    return t.contiguous().view(torch.uint8)


CASES = [
    # new tokens, cached lengths, kv heads, d, page, dtype, quant
    ([1], [1], 1, 64, 16, torch.bfloat16, False),
    ([1, 1, 1], [1000, 16, 17], 8, 128, 16, torch.bfloat16, True),
    ([5, 0, 33, 1], [700, 9, 33, 64], 2, 128, 32, torch.float16, False),
    ([100, 3, 1], [129, 300, 1], 5, 64, 64, torch.float16, True),
    ([257], [600], 3, 128, 128, torch.bfloat16, True),
    ([1] * 70, list(range(1, 71)), 1, 64, 256, torch.bfloat16, True),
    ([300, 400], [300, 1000], 16, 64, 16, torch.bfloat16, False),
    ([2000] + [1] * 40, [2000] + [3000] * 40, 2, 128, 64, torch.float16, True),
    # thousands of rows: several per warp, of sequences that begin and end among them
    ([0, 5001, 0, 0, 1, 2, 3, 0] + [3] * 700 + [6], [4, 5001, 7, 0, 900, 2, 33, 1] + [40] * 700 + [6], 2, 64, 16,
     torch.float16, True),
    ([12001, 1] + [7] * 1200, [12001, 3] + [7] * 1200, 1, 64, 32, torch.bfloat16, True),
    ([9001, 1, 0, 3000], [9100, 3, 9, 3001], 3, 128, 64, torch.bfloat16, False),
]


@pytest.mark.parametrize("new,lens,hk,d,page,dtype,quant", CASES)
def test_append_then_gather(new, lens, hk, d, page, dtype, quant):
    s = build(new, lens, hk, d, page, dtype, quant, seed=sum(lens) + d)
    before = [t.clone() for t in s["pages"]]
    append(s)
    table, at = s["table"].cpu(), 0
    touched = torch.zeros(s["pages"][0].shape[0], page, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(new, lens)):
        pg, slot = locate(table, b, torch.arange(m - n, m), page)
        touched[pg, slot] = True
    for x, pages, scales, old in ((s["k"], s["pages"][0], s["scales"][0], before[0]),
                                  (s["v"], s["pages"][1], s["scales"][1], before[1])):
        # slots that no row went to keep their bytes
        same = (bits(pages).view(*pages.shape[:3], -1) == bits(old).view(*pages.shape[:3], -1)).all(-1).cpu()
        assert torch.all(same | touched[:, None, :])
        at = 0
        for b, (n, m) in enumerate(zip(new, lens)):
            pg, slot = locate(table, b, torch.arange(m - n, m), page)
            rows = x[at:at + n].cpu()
            if quant:
                want, e = quantise_rows(rows)
                code = pages.float().cpu()[pg, :, slot].double()
                exp = bits(scales).view(scales.shape).cpu()[pg, :, slot].long() - 127
                assert torch.equal(exp, e) and torch.equal(code * torch.exp2(exp.double())[..., None], want)
            else:
                assert torch.equal(pages.cpu()[pg, :, slot], rows)
            at += n
    # the new rows read back: the values as held
    starts = s["seqlens"] - torch.tensor(new, dtype=torch.int32, device="cuda")
    ko, vo = api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], sum(new), starts=starts,
                              k_scales=s["scales"][0], v_scales=s["scales"][1], dtype=dtype)
    for got, x in ((ko, s["k"]), (vo, s["v"])):
        want = quantise_rows(x)[0] if quant else x.double().cpu()
        assert torch.equal(got.double().cpu(), want)
    assert api.get_status() == 0


@pytest.mark.parametrize("quant", [False, True])
def test_gather_ranges_padding_and_short_sequences(quant):
    """Windows of positions, rows past a sequence's length and rows behind the last sequence:
    those keep what the output held."""
    new, lens = [90, 200, 40], [90, 200, 40]
    s = build(new, lens, 2, 64, 32, torch.bfloat16, quant, seed=3)
    append(s)
    counts = [50, 33, 60]                                   # the last asks for more than there is
    starts = torch.tensor([30, 150, 0], dtype=torch.int32, device="cuda")
    cu = offsets(counts).cuda()
    out = [torch.full((150, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ko, vo = api.cache_gather(*s["pages"], s["table"], s["seqlens"], cu, 150, starts=starts, k_scales=s["scales"][0],
                              v_scales=s["scales"][1], k_out=out[0], v_out=out[1])
    assert ko is out[0] and vo is out[1]
    for got, x in ((ko.cpu(), s["k"].cpu()), (vo.cpu(), s["v"].cpu())):
        held = quantise_rows(x)[0] if quant else x.double()
        assert torch.equal(got[:50].double(), held[30:80])
        assert torch.equal(got[50:83].double(), held[90 + 150:90 + 183])
        assert torch.equal(got[83:123].double(), held[290:330])
        assert torch.all(got[123:] == 7.0)
    assert api.get_status() == 0


def test_e4m3_rows_at_the_borders():
    """Rows of zeros, of one magnitude, just at and above 448 times a power of two, of the type's
    extremes, ties, and with infinities and NaN."""
    for dtype in (torch.bfloat16, torch.float16):
        fin = torch.finfo(dtype)
        rows = torch.zeros(12, 1, 64)
        rows[1] = 3.5                                        # amax = 448 * 2^-7 exactly
        rows[2] = 3.5
        rows[2, 0, 5] = 3.516
        rows[3, 0, :3] = torch.tensor([fin.max, -fin.max, 1.0])
        rows[4] = fin.smallest_normal / 4                    # subnormal
        rows[5] = torch.arange(64) * 2.0 + 321.0             # ties of the coarsest steps
        rows[6] = torch.linspace(-1, 1, 64)
        rows[7, 0, 0], rows[7, 0, 1], rows[7, 0, 2] = float("inf"), float("-inf"), 2.0
        rows[8, 0, 0], rows[8, 0, 1] = float("nan"), 1.0
        rows[9] = float("nan")
        rows[10] = -0.0
        rows[11] = 2.0 ** torch.linspace(-20, 8, 64)
        x = rows.to(dtype)
        s = build([12], [12], 1, 64, 16, dtype, True, seed=1)
        append(s, k=x.cuda(), v=(-x).cuda())
        out = api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], 12, k_scales=s["scales"][0],
                               v_scales=s["scales"][1], dtype=dtype)
        for got, y in zip(out, (x, -x)):
            want = quantise_rows(y)[0]
            same = (got.double().cpu() == want) | (got.isnan().cpu() & want.isnan())
            assert same.all(), [(tuple(i), y[tuple(i)].item(), got[tuple(i)].item(), want[tuple(i)].item())
                                for i in (~same).nonzero().tolist()[:8]]
    assert api.get_status() == 0


def test_rows_behind_the_last_sequence_are_not_written():
    s = build([3, 2], [20, 2], 2, 128, 16, torch.bfloat16, False, seed=8)
    k = torch.randn(9, 2, 128, device="cuda").to(torch.bfloat16)     # four rows of padding
    append(s, k=k, v=k)
    written = torch.isfinite(s["pages"][0]).all(-1).all(1).sum().item()
    assert written == 5 and api.get_status() == 0


def test_bad_pages_and_positions_are_skipped_and_reported():
    """Page numbers and positions out of range leave the pools and the output alone; the other
    rows are written and read."""
    s = build([4, 4], [40, 4], 1, 64, 16, torch.bfloat16, False, seed=9)
    good = s["table"].clone()
    for bad_page in (-1, s["pages"][0].shape[0], 2 ** 31 - 1):
        s["table"].copy_(good)
        s["table"][0, 2] = bad_page                           # positions 36..39 of sequence 0
        for t in s["pages"]:
            t.fill_(float("nan"))
        append(s)
        assert api.get_status_site() == (9, 41)
        assert torch.isfinite(s["pages"][0]).all(-1).sum().item() == 4
        out = [torch.full((8, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], 8, starts=s["seqlens"] - 4, k_out=out[0],
                         v_out=out[1])
        assert api.get_status_site() == (9, 42)
        assert torch.all(out[0][:4] == 5.0) and torch.equal(out[0][4:], s["k"][4:])
    s["table"].copy_(good)
    s["seqlens"][1] = 2                                       # shorter than its new tokens
    append(s)
    assert api.get_status() == 9
    s["seqlens"][1] = 10 ** 6                                 # past the table
    append(s)
    assert api.get_status() == 9 and api.get_status() == 0


def test_append_captured_and_replayed_as_the_cache_grows():
    s = build([1, 1], [100, 31], 2, 128, 32, torch.float16, True, seed=10)
    append(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        append(s)
    s["qkv"].copy_(torch.randn_like(s["qkv"]))
    s["seqlens"] -= 1
    g.replay()
    ko, _ = api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], 2, starts=s["seqlens"] - 1,
                             k_scales=s["scales"][0], v_scales=s["scales"][1], dtype=torch.float16)
    assert torch.equal(ko.double().cpu(), quantise_rows(s["k"])[0]) and api.get_status() == 0


def test_cache_refusals():
    s = build([2], [20], 2, 64, 16, torch.bfloat16, False, seed=11)
    append(s, k=s["k"][:0], v=s["v"][:0])                     # nothing to write
    for kw, err in ((dict(k=s["k"].half()), TypeError), (dict(k=s["k"][:, :1]), ValueError),
                    (dict(v_pages=s["pages"][1][:1]), ValueError), (dict(page_table=s["table"].long()), ValueError),
                    (dict(seqlens=s["seqlens"].long()), ValueError), (dict(cu_q=s["cu"][:1]), ValueError),
                    (dict(k_scales=s["cu"]), ValueError), (dict(k=s["k"].transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            append(s, **kw)
    q = build([2], [20], 2, 64, 16, torch.bfloat16, True, seed=11)
    with pytest.raises(ValueError):
        append(q, k_scales=None)
    odd = torch.zeros(2, 2, 72, dtype=torch.bfloat16, device="cuda")[..., 1:65]    # rows not 16-byte aligned
    with pytest.raises(api.FAError):
        append(s, k=odd)
    with pytest.raises(TypeError):
        api.cache_gather(*q["pages"], q["table"], q["seqlens"], q["cu"], 2, k_scales=q["scales"][0],
                         v_scales=q["scales"][1], dtype=torch.float32)
    with pytest.raises(ValueError):
        api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], -1)
    three = [torch.zeros(4, 2, 48, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]    # pages of 48
    with pytest.raises(api.FAError):
        api.cache_gather(*three, s["table"], s["seqlens"], s["cu"], 2)


def test_cache_buffers_that_overlap():
    s = build([2], [20], 2, 64, 16, torch.bfloat16, True, seed=12)
    for kw in (dict(v_pages=s["pages"][0]), dict(v_scales=s["scales"][0])):
        with pytest.raises(ValueError):
            append(s, **kw)
    out = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for k_out, v_out in ((out[:2], out[1:]), (out[:2], out[:2])):
        with pytest.raises(ValueError):
            api.cache_gather(*s["pages"], s["table"], s["seqlens"], s["cu"], 2, k_scales=s["scales"][0],
                             v_scales=s["scales"][1], k_out=k_out, v_out=v_out)
    assert api.get_status() == 0
