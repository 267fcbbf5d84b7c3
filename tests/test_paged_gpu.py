"""Attention over a paged cache through fa_paged, against dense attention in fp64.

Tolerance of O, per element.  The softmax weights are rounded to the 16-bit type, u = eps / 2
relative (fp16: or 2^-25 where subnormal), after an error eta = 2^-14 from fp32 scores (up to
128 products of size |q k|, |score| < 2^5, rounded at 2^-24) and the 2^-22 exponential.  bf16
divides by the sum of the rounded weights, so an error of a weight moves O by its distance to
that value row: at most (u + eta) sum_j w_j |v_j - O| / (1 - u - eta); fp16 divides by the fp32
sum: (u + eta) sum_j w_j |v_j|, plus 2^-25 per key.  Then the output rounds (u |O|).  fp32 sums
over the keys add at most 2^-17 max|v|.  LSE: eta, and 2^-20 relative.

e4m3 pages: a weight is an fp16 value, kept to 9 bits for bf16 queries (u = 2^-9) and whole for
fp16 (u = 2^-11), and loses what lies under 2^-16 / 2^7 = 2^-23 of the largest weight (times a
value of up to 2 max|v|, by the scales' powers of two); the fp32 sum divides.  Query pieces end
at 2^-10 with a row maximum of at least 224: 2^-17.8 of it per element, which moves a score by up
to 2^-17.8 scale max|q| sum|k| < 2^-12.5 at these sizes, so eta = 2^-12."""
import math

import pytest
import torch

from exact_io_aware_93_b200 import api
from tests.paged import locate, offsets, page_tables, quantise_rows

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def build(new, lens, h, hk, d, page, dtype, quant, seed, window=-1, spread=1.0):
    """A batch with its paged cache.  Everything that no token sees holds NaN: slots past a
    length, pages of nobody, positions and pages a window has left behind (those pages' table
    entries are -1)."""
    g = torch.Generator().manual_seed(seed)
    table, pool = page_tables(lens, page, g)
    s = dict(new=new, lens=lens, window=window, h=h, hk=hk)
    s["q"] = (torch.randn(sum(new), h, d, generator=g) * spread).to(dtype)
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32)
    s["cu"] = offsets(new)
    shape = (pool, hk, page, d)
    s["values"] = []
    pages, scales = [], []
    for _ in "kv":
        x = torch.full(shape, float("nan"), dtype=dtype)
        e = torch.full(shape[:3], 255, dtype=torch.uint8)
        vals = []
        for b, (n, m) in enumerate(zip(new, lens)):
            rows = torch.randn(m, hk, d, generator=g).to(dtype)
            if quant:
                held, exp = quantise_rows(rows)
            else:
                held, exp = rows.double(), None
            first = max(0, m - n - window) if window >= 0 else 0
            pos = torch.arange(first, m)
            pg, slot = locate(table, b, pos, page)
            x[pg, :, slot] = (held[first:] / torch.exp2(exp[first:].double())[..., None] if quant else held[first:]).to(dtype)
            if quant:
                e[pg, :, slot] = (exp[first:] + 127).to(torch.uint8)
            vals.append(held)
        pages.append((x.float().to(torch.float8_e4m3fn) if quant else x).cuda())
        scales.append(e.view(torch.float8_e8m0fnu).cuda() if quant else None)
        s["values"].append(vals)
    for b, (n, m) in enumerate(zip(new, lens)):
        if window >= 0:
            table[b, :max(0, m - n - window) // page] = -1
    s["pages"], s["scales"], s["table"] = pages, scales, table.cuda()
    for k in ("q", "seqlens", "cu"):
        s[k] = s[k].cuda()
    return s


def attend(s, causal=True, **kw):
    a = dict(q=s["q"], k_pages=s["pages"][0], v_pages=s["pages"][1], page_table=s["table"], seqlens=s["seqlens"],
             cu_q=s["cu"], max_q=max(max(s["new"]), 1), causal=causal, window=None if s["window"] < 0 else s["window"],
             k_scales=s["scales"][0], v_scales=s["scales"][1])
    a.update(kw)
    return api.paged_attention(**a)


def check(s, o, lse, causal=True, scale=None, q=None):
    q = s["q"] if q is None else q
    d, dtype = q.shape[-1], q.dtype
    scale = d ** -0.5 if scale is None else scale
    quant = s["scales"][0] is not None
    out_u = torch.finfo(dtype).eps / 2
    u, eta = (out_u, 2.0 ** -14) if not quant else (2.0 ** -9 if dtype == BF else out_u, 2.0 ** -12)
    at = 0
    group = s["h"] // s["hk"]
    for b, (n, m) in enumerate(zip(s["new"], s["lens"])):
        if n == 0:
            continue
        k, v = (s["values"][i][b].cuda().transpose(0, 1).repeat_interleave(group, 0) for i in range(2))   # [H, m, d]
        x = torch.matmul(q[at:at + n].double().transpose(0, 1), k.transpose(1, 2)) * scale            # [H, n, m]
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        key = torch.arange(m, device="cuda")[None]
        seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
        if causal:
            seen = key <= pos
            if s["window"] >= 0:
                seen = seen & (key >= pos - s["window"])
        x = x.masked_fill(~seen, -math.inf)
        none = ~seen.any(-1)
        want_l = torch.logsumexp(x, -1) if m else torch.full((s["h"], n), -math.inf, dtype=torch.float64, device="cuda")
        w = torch.exp(x - want_l[..., None]).masked_fill(~seen, 0.0).masked_fill(none[:, None], 0.0)
        want = torch.matmul(w, v)
        tol = torch.zeros_like(want)
        if m:
            top = v.abs().amax()
            for r in range(0, n, 64):                        # sum_j w_j |v_j - O|, a block of rows at a time
                wr = w[:, r:r + 64]
                if quant or dtype == torch.float16:
                    lost = m * (2.0 ** -22 if quant else 2.0 ** -25) * top
                    tol[:, r:r + 64] = torch.matmul(wr, v.abs()) + lost / u
                else:
                    for c in range(0, d, 16):
                        far = (v[:, None, :, c:c + 16] - want[:, r:r + 64, None, c:c + 16]).abs()
                        tol[:, r:r + 64, c:c + 16] = (wr[..., None] * far).sum(2)
            tol = (u + eta) * tol / (1 - u - eta) + 2.0 ** -17 * top
        tol = tol + out_u * (want.abs() + tol) + 2.0 ** -25
        got = o[at:at + n].double().transpose(0, 1)
        err = (got - want).abs()
        assert torch.all(err <= tol), (b, (err - tol).max().item(), (err / tol).max().item())
        gl = lse[:, at:at + n].double()
        assert torch.equal(torch.isneginf(gl), none.expand_as(gl))
        keep = ~none.expand_as(gl)
        assert torch.all((gl - want_l)[keep].abs() <= eta + 2.0 ** -20 * want_l.abs()[keep]), b
        at += n


CASES = [
    # new tokens, lengths, heads, kv heads, d, page, dtype, e4m3, causal, window
    ([1], [1], 1, 1, 64, 16, BF, False, True, -1),                           # one key
    ([1, 1, 1], [1000, 1, 517], 8, 2, 128, 16, BF, False, True, -1),          # decoding, ragged
    ([1] * 5, [130, 128, 129, 127, 2000], 32, 8, 128, 64, BF, True, True, -1),
    ([1] * 5, [130, 128, 129, 127, 2000], 8, 8, 64, 32, FP, True, True, -1),
    ([1, 0, 1], [700, 33, 0], 4, 4, 64, 128, FP, False, True, -1),            # nothing to do, and an empty cache
    ([3, 2], [700, 2], 4, 4, 64, 256, BF, False, True, -1),                   # as many tokens as keys
    ([3, 2], [2, 900], 4, 2, 64, 16, BF, False, True, -1),                    # more tokens than keys
    ([4, 4], [900, 300], 8, 1, 128, 32, FP, False, False, -1),                # not causal, 32 rows
    ([8, 5], [1300, 129], 16, 2, 128, 64, BF, False, True, 100),              # 64 rows, window
    ([5, 5], [1300, 600], 6, 2, 128, 16, FP, True, True, 100),                # 15 rows of e4m3, window
    ([1, 1], [1300, 600], 16, 1, 64, 16, BF, True, True, 0),                  # window 0: the key itself
    ([1, 1], [5000, 300], 128, 1, 128, 64, BF, False, True, -1),              # 128 heads share one
    ([16, 1], [700, 650], 8, 2, 128, 32, BF, False, True, 255),
    ([200], [200], 4, 4, 128, 64, BF, False, True, -1),                       # a prompt from its start
    ([300, 1, 1, 77], [900, 1200, 1, 77], 8, 2, 128, 16, BF, False, True, -1),   # mixed
    ([300, 1, 1, 77], [900, 1200, 1, 77], 8, 2, 128, 16, BF, True, True, -1),
    ([300, 1, 129], [900, 1200, 640], 4, 2, 64, 32, FP, True, False, -1),
    ([500, 130], [1500, 130], 6, 2, 64, 128, FP, False, True, 77),            # groups of 3: 126 rows a tile
    ([260, 3], [1030, 700], 5, 1, 128, 256, BF, False, True, 300),            # groups of 5
    ([260, 0, 3], [1030, 40, 700], 7, 1, 64, 64, BF, True, True, 129),
    ([400], [300], 2, 1, 64, 16, BF, False, True, -1),                        # the first tokens see nothing
    ([1] * 40, [17 * i + 1 for i in range(40)], 4, 2, 64, 16, BF, False, True, -1),
    ([2] * 70, [30 * i + 2 for i in range(70)], 16, 4, 128, 32, FP, True, True, 200),
    ([40] * 3, [100, 64, 40], 3, 3, 128, 16, FP, False, True, -1),            # 40 rows: one tile
    ([90] * 3, [300, 164, 140], 3, 3, 128, 16, FP, True, True, 30),
    ([2, 1, 2], [3000, 130, 2], 16, 4, 128, 64, BF, True, True, -1),          # 8 rows of four lanes
    ([1, 1, 1], [1, 4097, 128], 5, 1, 64, 16, BF, True, True, -1),
    ([1] * 9, [513 * i + 1 for i in range(9)], 8, 8, 128, 128, FP, True, False, -1),
    ([1] * 3, [2000] * 3, 24, 2, 128, 32, BF, True, True, -1),                # 12 rows of e4m3
    ([1] * 3, [2000] * 3, 40, 2, 64, 256, BF, True, True, 900),               # 20 rows of e4m3
    ([70, 1, 1, 1], [2000, 700, 1500, 3000], 8, 2, 64, 64, BF, True, True, -1),
    ([70, 65, 1, 64], [4000, 700, 1500, 64], 2, 2, 128, 128, FP, False, True, -1),
]


@pytest.mark.parametrize("new,lens,h,hk,d,page,dtype,quant,causal,window", CASES)
def test_paged_attention(new, lens, h, hk, d, page, dtype, quant, causal, window):
    s = build(new, lens, h, hk, d, page, dtype, quant, seed=sum(lens) + h + d, window=window)
    o, lse = attend(s, causal)
    torch.cuda.synchronize()
    assert api.get_status_site() == (0, 0)
    check(s, o, lse, causal)
