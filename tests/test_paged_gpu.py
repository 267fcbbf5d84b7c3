"""Attention over a paged cache through fa_paged, against dense attention in fp64.

Tolerance of O, per element.  The softmax weights are rounded to the 16-bit type, u = eps / 2
relative (fp16: or 2^-25 where subnormal), after an error eta = 2^-14 from fp32 scores (up to
128 products of size |q k|, |score| < 2^5, rounded at 2^-24) and the 2^-22 exponential.  bf16
divides by the sum of the rounded weights, so an error of a weight moves O by its distance to
that value row: at most (u + eta) sum_j w_j |v_j - O| / (1 - u - eta); fp16 divides by the fp32
sum: (u + eta) sum_j w_j |v_j|, plus 2^-25 per key.  Then the output rounds (u |O|).  fp32 sums
over the keys add at most 2^-17 max|v|.  LSE: eta, and 2^-20 relative.

e4m3 pages: a weight is an fp16 value, kept to 9 bits for bf16 queries (u = 2^-9) and whole for
fp16 (u = 2^-11).  It is cut off at 2^-16 / 2^13 = 2^-29 of the reference weight, which is at most
the largest, with few rows, and rounded by fp16's smallest step at 2^-25 of it in tiles of 128 (times
a value of up to 2 max|v|, by the scales' powers of two); the fp32 sum divides.  Query pieces end at
2^-10 with a row maximum of at least 224: 2^-17.8 of it per element, which moves a score by up to
2^-17.8 scale max|q| sum|k| < 2^-12.5 at these sizes, so eta = 2^-12."""
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
                    lost = m * (2.0 ** -24 if quant else 2.0 ** -25) * top
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


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    """Random shapes, kinds and lengths of everything the entry point takes."""
    import random
    rng = random.Random(4000 + seed)
    hk = rng.choice([1, 1, 2, 3, 4])
    h = hk * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    kind = rng.choice(["one", "few", "chunk", "mixed"])
    page = rng.choice([16, 32, 64, 128, 256])
    new, lens = [], []
    for _ in range(rng.randint(1, 9)):
        n = {"one": 1, "few": rng.randint(1, 7), "chunk": rng.randint(1, 300),
             "mixed": rng.choice([0, 1, 1, 2, rng.randint(1, 200)])}[kind]
        m = rng.choice([n, rng.randint(1, 1500), rng.randint(1, 1500), page * rng.randint(1, 4)])
        new.append(n)
        lens.append(m)
    if sum(new) == 0:
        new[0], lens[0] = 1, max(lens[0], 1)
    causal = rng.random() < 0.8
    window = rng.choice([-1, -1, 0, 17, 127, 400]) if causal else -1
    s = build(new, lens, h, hk, rng.choice([64, 128]), page, rng.choice([BF, FP]), rng.random() < 0.5, seed=seed,
              window=window)
    o, lse = attend(s, causal, max_q=max(new) + rng.choice([0, 0, 1, 60]))
    torch.cuda.synchronize()
    assert api.get_status_site() == (0, 0)
    check(s, o, lse, causal)


KINDS = [  # batches that take the few-rows kernel, the tiles, and both
    ([1] * 6, [700, 30, 129, 1500, 64, 1]),
    ([50, 41], [300, 900]),
    ([1, 130, 1, 1], [700, 300, 129, 2000]),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", KINDS)
def test_strides_given_buffers_and_padding(new, lens, quant):
    """q as a slice of a fused projection, buffers of the caller's, rows behind the last sequence
    and guard zones around everything that is written."""
    s = build(new, lens, 8, 2, 128, 32, BF, quant, seed=5)
    want, want_l = attend(s)
    T, pad = sum(new), 37
    fused = torch.full((T + pad, 12, 128), float("nan"), dtype=BF, device="cuda")
    fused[:T, 2:10] = s["q"]
    guard = 1024
    nbytes = api.paged_workspace_size(fused[:, 2:10], s["pages"][0], s["table"], max(new))
    flat = torch.full((2 * guard + (T + pad) * 1024,), 3.0, dtype=BF, device="cuda")
    flat_l = torch.full((2 * guard + 8 * (T + pad),), 5.0, device="cuda")
    ws = torch.full((2 * guard + nbytes,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN everywhere
    out = flat[guard:-guard].view(T + pad, 8, 128)
    lse = flat_l[guard:-guard].view(8, T + pad)
    o2, l2 = attend(s, q=fused[:, 2:10], out=out, lse=lse, workspace=ws[guard:guard + nbytes])
    torch.cuda.synchronize()
    assert api.get_status_site() == (0, 0) and o2 is out and l2 is lse
    assert torch.equal(out[:T], want) and torch.equal(lse[:, :T], want_l)
    assert torch.all(out[T:] == 3.0) and torch.all(lse[:, T:] == 5.0)
    for t, v in ((flat, 3.0), (flat_l, 5.0), (ws, 0xFF)):
        assert torch.all(t[:guard] == v) and torch.all(t[-guard:] == v)
    with pytest.raises(api.FAError) as e:
        attend(s, workspace=ws[guard:guard + nbytes // 512 * 256])
    assert e.value.status == 7


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", KINDS)
def test_same_bits_again(new, lens, quant):
    s = build(new, lens, 8, 2, 64, 64, FP, quant, seed=6)
    o, lse = attend(s)
    for fill in (0x00, 0x7F, 0xFF):
        ws = torch.full((api.paged_workspace_size(s["q"], s["pages"][0], s["table"], max(new)),), fill, dtype=torch.uint8,
                        device="cuda")
        o2, l2 = attend(s, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert api.get_status() == 0


@pytest.mark.parametrize("quant", [False, True])
def test_captured_graph_replayed_as_the_batch_changes(quant):
    """One capture serves other lengths, other tokens per sequence and other pages, within B, T and
    max_q; a second graph with the same workspace replays after it."""
    batches = [build(n, m, 8, 2, 128, 32, BF, quant, seed=7) for n, m in
               (([1, 60, 3], [900, 300, 200]), ([64, 0, 0], [1000, 3, 2]), ([0, 1, 1], [0, 1200, 5]))]
    pool = max(b["pages"][0].shape[0] for b in batches)
    width = max(b["table"].shape[1] for b in batches)
    first = batches[0]
    live = dict(first)
    live["pages"] = [torch.zeros((pool, *first["pages"][0].shape[1:]), dtype=first["pages"][0].dtype, device="cuda")
                     for _ in "kv"]
    if quant:
        live["scales"] = [torch.zeros((pool, *first["scales"][0].shape[1:]), dtype=torch.uint8, device="cuda")
                          .view(torch.float8_e8m0fnu) for _ in "kv"]
    live["table"] = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    live["q"] = torch.zeros(64, 8, 128, dtype=BF, device="cuda")
    live["seqlens"], live["cu"] = first["seqlens"].clone(), first["cu"].clone()
    ws = torch.empty(api.paged_workspace_size(live["q"], live["pages"][0], live["table"], 64), dtype=torch.uint8,
                     device="cuda")
    out = [torch.empty(64, 8, 128, dtype=BF, device="cuda") for _ in range(2)]
    lse = [torch.empty(8, 64, device="cuda") for _ in range(2)]

    def fill(b):
        for x, y in zip(live["pages"], b["pages"]):
            x[:y.shape[0]].view(torch.uint8).copy_(y.view(torch.uint8))
        if quant:
            for x, y in zip(live["scales"], b["scales"]):
                x[:y.shape[0]].view(torch.uint8).copy_(y.view(torch.uint8))
        live["table"].fill_(-1)
        live["table"][:, :b["table"].shape[1]] = b["table"]
        live["q"].fill_(float("nan"))
        live["q"][:b["q"].shape[0]] = b["q"]
        live["seqlens"].copy_(b["seqlens"])
        live["cu"].copy_(b["cu"])
    fill(first)
    graphs = []
    for i in range(2):
        attend(live, max_q=64, out=out[i], lse=lse[i], workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(live, max_q=64, out=out[i], lse=lse[i], workspace=ws)
        graphs.append(g)
    for b in batches[1:] + batches[:1]:
        fill(b)
        for i in range(2):
            out[i].fill_(-2.0)
            lse[i].fill_(-2.0)
            graphs[i].replay()
        torch.cuda.synchronize()
        assert api.get_status_site() == (0, 0)
        T = sum(b["new"])
        check(b, out[0], lse[0])
        assert torch.all(out[0][T:] == -2.0) and torch.all(lse[0][:, T:] == -2.0)
        assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", KINDS)
def test_captured_behind_copies_and_other_streams(new, lens, quant):
    """In a graph behind a memory copy, behind a kernel, and where two streams join: the call waits
    for what it reads each time."""
    s = build(new, lens, 8, 2, 128, 32, BF, quant, seed=18)
    want, want_l = attend(s)
    torch.cuda.synchronize()
    live = dict(s, q=torch.zeros_like(s["q"]), seqlens=torch.zeros_like(s["seqlens"]))
    side = torch.cuda.Stream()
    big = torch.empty(1 << 26, device="cuda")
    graphs = []
    for before in ("copy", "kernel", "join"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            main = torch.cuda.current_stream()
            if before == "join":
                side.wait_stream(main)
                with torch.cuda.stream(side):
                    big.add_(1.0)
                    live["seqlens"].copy_(s["seqlens"])
            big.mul_(0.5)                                    # long enough to be still running
            if before != "join":
                live["seqlens"].copy_(s["seqlens"])
            if before == "copy":
                live["q"].copy_(s["q"])
            else:
                torch.add(s["q"], 0.0, out=live["q"])
            if before == "join":
                main.wait_stream(side)
            out = attend(live)
            live["q"].zero_()
            live["seqlens"].zero_()
        graphs.append((g, out))
    for _ in range(2):
        for g, (o, lse) in graphs:
            o.fill_(-1.0)
            g.replay()
            torch.cuda.synchronize()
            assert api.get_status_site() == (0, 0)
            assert torch.equal(o, want) and torch.equal(lse, want_l)


def test_two_streams_at_once():
    """Calls in flight on two streams, and on one that is not the tensors' own, each with its own
    workspace."""
    a = build([1] * 8, [3000 + 100 * i for i in range(8)], 16, 4, 128, 64, BF, True, seed=8)
    b = build([200, 1, 1], [2500, 1900, 40], 16, 4, 128, 16, FP, True, seed=9)
    want = [attend(a), attend(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(attend(s))
    torch.cuda.synchronize()
    assert api.get_status_site() == (0, 0)
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_shared_pages_and_uint8_scales():
    """Sequences that share the pages of a prefix give what copies of it give; scales may be uint8."""
    s = build([2, 2, 2], [300, 300, 300], 4, 2, 64, 16, BF, True, seed=10)
    s["q"][2:4] = s["q"][0:2]
    s["q"][4:6] = s["q"][0:2]
    s["table"][1] = s["table"][0]
    s["table"][2] = s["table"][0]
    o, lse = attend(s, k_scales=s["scales"][0].view(torch.uint8), v_scales=s["scales"][1].view(torch.uint8))
    assert api.get_status() == 0
    assert torch.equal(o[0:2], o[2:4]) and torch.equal(o[0:2], o[4:6]) and torch.equal(lse[:, :2], lse[:, 4:])


@pytest.mark.parametrize("dtype,quant,rows", [(BF, True, 1), (FP, True, 1), (BF, True, 40), (FP, True, 40), (FP, False, 1)])
def test_long_tail_of_small_weights(dtype, quant, rows):
    """One key takes nearly all of the softmax; thousands of others, 2^-18 of it each, still add up:
    with values 0 for it and 1 for them O is their share."""
    m, c = 16384, 18.0 * math.log(2.0)
    s = build([rows], [m], 1, 1, 64, 64, dtype, quant, seed=11)
    k = torch.zeros(m, 1, 64, dtype=dtype, device="cuda")
    k[:, 0, 0] = -1.0
    k[3, 0, 0] = 0.0
    v = torch.ones(m, 1, 64, dtype=dtype, device="cuda")
    v[3] = 0.0
    api.cache_append(k, v, *s["pages"], s["table"], s["seqlens"], torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                     k_scales=s["scales"][0], v_scales=s["scales"][1])
    s["q"].zero_()
    s["q"][:, 0, 0] = 16.0
    o, lse = attend(s, causal=False, scale=c / 16.0)
    assert api.get_status() == 0
    share = (m - 1) * math.exp(-c) / (1.0 + (m - 1) * math.exp(-c))       # 0.0588
    # a weight: 2^-9 (bf16) or 2^-11 of itself, or 2^-25 of the largest, 2^-7 of itself, and equal
    # weights round alike; fp32 scores of 12.5: 2^-20; then the output's rounding
    rel = (2.0 ** -7 if rows > 32 or not quant else 2.0 ** -9) + 2.0 ** -20 + torch.finfo(dtype).eps / 2
    assert (o.double() / share - 1.0).abs().max().item() <= rel
    assert (lse.double() - math.log1p((m - 1) * math.exp(-c))).abs().max().item() <= 2.0 ** -14


@pytest.mark.parametrize("dtype,quant,rows", [(FP, False, 1), (FP, False, 40), (FP, True, 40), (BF, True, 40)])
def test_little_weights_of_a_long_cache_keep_their_sum(dtype, quant, rows):
    """A key of weight 1 in each of the first two tiles and thousands of 2^-26.6 each behind them, every
    key/value head in one run of an SM: with values 0 for the two and 1 for the others O is the others'
    share, 2^-14.6.  A weight is kept to 2^-25 / 2^7 = 2^-32 of the reference: 2^-5.4 of itself; the
    output to fp16's smallest half step, 2^-25, or 2^-9 of itself."""
    m, c = 8192, 26.6 * math.log(2.0)
    hk = torch.cuda.get_device_properties(0).multi_processor_count
    page = 256
    table = torch.arange(m // page, dtype=torch.int32, device="cuda")[None]
    kind = torch.float8_e4m3fn if quant else dtype
    pages = [torch.zeros(m // page, hk, page, 64, dtype=kind, device="cuda") for _ in "kv"]
    scales = [torch.full((m // page, hk, page), 127, dtype=torch.uint8, device="cuda") if quant else None for _ in "kv"]
    k = torch.zeros(m, 1, 64, dtype=dtype, device="cuda")
    k[:, 0, 0] = -1.0
    k[[3, 131]] = 0.0
    v = torch.ones(m, 1, 64, dtype=dtype, device="cuda")
    v[[3, 131]] = 0.0
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([m], [0, m]))
    api.cache_append(k.expand(m, hk, 64), v.expand(m, hk, 64), *pages, table, lens, cu, k_scales=scales[0],
                     v_scales=scales[1])
    q = torch.zeros(1, hk * rows, 64, dtype=dtype, device="cuda")
    q[:, :, 0] = 16.0
    o, lse = api.paged_attention(q, *pages, table, lens, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1,
                                 scale=c / 16.0, k_scales=scales[0], v_scales=scales[1])
    assert api.get_status() == 0
    tail = (m - 2) * math.exp(-c)
    share = tail / (2.0 + tail)
    tol = share * 2.0 ** -5.4 * (1 + 2.0 ** -10) + max(2.0 ** -25, share * torch.finfo(dtype).eps / 2)
    assert (o.double() - share).abs().max().item() <= tol
    assert (lse.double() - math.log(2.0 + tail)).abs().max().item() <= 2.0 ** -14


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,lens", KINDS)
def test_bad_page_numbers_of_an_e4m3_cache_read_as_zeros(new, lens, dtype):
    """What a page of zero codes with scale 1 gives, bit for bit."""
    s = build(new, lens, 8, 2, 128, 32, dtype, True, seed=15)
    at = s["table"][-1, 0].item() if lens[-1] < 200 else s["table"][-1, 3].item()
    col = 0 if lens[-1] < 200 else 3
    for x, e in zip(s["pages"], s["scales"]):
        x.view(torch.uint8)[at] = 0
        e.view(torch.uint8)[at] = 127
    want, want_l = attend(s)
    assert api.get_status() == 0
    for x, e in zip(s["pages"], s["scales"]):     # what must not be read
        x.view(torch.uint8)[at] = 0x7F
        e.view(torch.uint8)[at] = 255
    for bad in (-1, s["pages"][0].shape[0]):
        s["table"][-1, col] = bad
        o, lse = attend(s)
        assert api.get_status_site() == (9, 44)
        assert torch.equal(o, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_queries_stay_in_their_row(new, lens, quant, value):
    """A query that is not finite changes no bit of another's row; a NaN makes its own NaN."""
    s = build(new, lens, 8, 2, 128, 32, BF, quant, seed=16)
    want, want_l = attend(s)
    s["q"] = s["q"].clone()
    s["q"][0, 1, 5] = value
    s["q"][-1, 7, 0] = value
    o, lse = attend(s)
    assert api.get_status() == 0
    hit = torch.zeros(o.shape[:2], dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[-1, 7] = True
    if math.isnan(value):
        assert torch.all(torch.isnan(o[hit])) and torch.all(torch.isnan(lse.t()[hit]))
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse.t()[~hit], want_l.t()[~hit])


def test_outputs_apart_from_what_is_read():
    s = build([2, 1], [50, 20], 4, 2, 64, 16, BF, False, seed=17)
    flat = s["pages"][0].view(-1)
    for kw in (dict(out=s["q"]), dict(out=flat[:3 * 4 * 64].view(3, 4, 64)), dict(lse=flat[:24].view(torch.float32).view(4, 3)),
               dict(workspace=s["q"])):
        with pytest.raises(ValueError):
            attend(s, **kw)
    assert api.get_status() == 0


def test_bad_plans_are_reported_and_skip_their_access():
    """Offsets, lengths and page numbers out of range: recorded, and everything else computed."""
    s = build([1, 1, 1], [500, 400, 300], 8, 2, 128, 32, BF, False, seed=12)
    good_o, good_l = attend(s)
    table, lens, cu = s["table"].clone(), s["seqlens"].clone(), s["cu"].clone()
    for bad in (-1, -2 ** 31, s["pages"][0].shape[0], 2 ** 31 - 1):
        s["table"].copy_(table)
        s["table"][1, 3] = bad
        o, lse = attend(s)
        assert api.get_status_site() == (9, 44)
        assert torch.equal(o[[0, 2]], good_o[[0, 2]]) and torch.equal(lse[:, [0, 2]], good_l[:, [0, 2]])
    s["table"].copy_(table)
    for bad in (-5, 10 ** 6, 2 ** 31 - 1):
        s["seqlens"].copy_(lens)
        s["seqlens"][1] = bad
        o, lse = attend(s)
        assert api.get_status() == 9
        assert torch.equal(o[[0, 2]], good_o[[0, 2]])
    s["seqlens"].copy_(lens)
    for bad in ([0, 2, 1, 3], [0, 1, 2, 9], [-4, 1, 2, 3], [0, 2 ** 31 - 1, 2, 3], [5, 5, 5, 5]):
        s["cu"].copy_(torch.tensor(bad, dtype=torch.int32))
        flat = torch.full((5, 8, 128), 3.0, dtype=BF, device="cuda")
        attend(s, out=flat[1:4])
        st = api.get_status_site()
        assert st == (9, 43) and torch.all(flat[0] == 3.0) and torch.all(flat[4] == 3.0)
    s["cu"].copy_(cu)
    o, lse = attend(s)
    assert torch.equal(o, good_o) and api.get_status() == 0


def test_refusals():
    s = build([2, 1], [50, 20], 4, 2, 64, 16, BF, True, seed=13)
    for kw, err in ((dict(q=s["q"].float()), TypeError), (dict(q=s["q"][0]), ValueError), (dict(q=s["q"].cpu()), ValueError),
                    (dict(q=s["q"][:, :3]), ValueError), (dict(q=s["q"][..., :32]), ValueError),
                    (dict(q=s["q"].transpose(1, 2)), ValueError), (dict(k_scales=None), ValueError),
                    (dict(v_scales=s["scales"][1][:1]), ValueError), (dict(page_table=s["table"][:1]), ValueError),
                    (dict(cu_q=s["cu"].long()), ValueError), (dict(seqlens=s["seqlens"][:1]), ValueError),
                    (dict(out=s["q"][:2]), ValueError), (dict(lse=torch.empty(4, 4, device="cuda")), ValueError),
                    (dict(workspace=torch.empty(1 << 20)), ValueError), (dict(max_q=2 ** 40), ValueError),
                    (dict(max_q=0), api.FAError), (dict(window=-3), api.FAError), (dict(scale=-1.0), api.FAError),
                    (dict(causal=False, window=5), api.FAError),
                    (dict(k_pages=s["pages"][0][:0], v_pages=s["pages"][1][:0]), ValueError)):
        with pytest.raises(err):
            attend(s, **kw)
    with pytest.raises(TypeError):
        attend(build([2], [50], 4, 2, 64, 16, BF, False, seed=13), q=s["q"][:2].half())
    o, lse = attend(s, q=s["q"][:0])                                   # no tokens: nothing to do
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    torch.cuda.synchronize()
    assert api.get_status() == 0


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of the pool (and 2^31 elements) are written, read back and attended."""
    hk, page, d, pool = 8, 256, 128, 8400                              # 2.2e9 elements each
    pages = [torch.empty(pool, hk, page, d, dtype=BF, device="cuda") for _ in "kv"]
    n, m = 3, 600
    g = torch.Generator().manual_seed(14)
    table = torch.tensor([[8399, 8398, 8250]], dtype=torch.int32, device="cuda")
    x = [torch.randn(m, hk, d, generator=g).to(BF).cuda() for _ in "kv"]
    lens = torch.tensor([m], dtype=torch.int32, device="cuda")
    api.cache_append(*x, *pages, table, lens, torch.tensor([0, m], dtype=torch.int32, device="cuda"))
    back = api.cache_gather(*pages, table, lens, torch.tensor([0, m], dtype=torch.int32, device="cuda"), m)
    assert torch.equal(back[0], x[0]) and torch.equal(back[1], x[1])
    s = dict(new=[n], lens=[m], window=-1, h=16, hk=hk, q=torch.randn(n, 16, d, generator=g).to(BF).cuda(), pages=pages,
             scales=[None, None], table=table, seqlens=lens, cu=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
             values=[[t.double().cpu()] for t in x])
    o, lse = attend(s)
    assert api.get_status() == 0
    check(s, o, lse)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,lens", KINDS)
@pytest.mark.parametrize("which", [0, 1])
def test_nan_scales_reach_the_rows_that_see_them(new, lens, dtype, which):
    """A scale byte of 255 makes its row NaN: every token of the sequence sees it, and other sequences
    keep their bits.  A NaN value changes no log-sum."""
    s = build(new, lens, 8, 2, 128, 32, dtype, True, seed=19)
    want, want_l = attend(s)
    hit = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    for b in range(2 if new[1] > 1 else 1):
        pg, slot = s["table"][b, 0].item(), 5 + b
        s["scales"][which].view(torch.uint8)[pg, :, slot] = 255
        hit[s["cu"][b]:s["cu"][b + 1]] = True
    o, lse = attend(s)
    assert api.get_status() == 0
    assert torch.all(torch.isnan(o[hit])) and torch.equal(o[~hit], want[~hit])
    assert torch.equal(lse[:, ~hit], want_l[:, ~hit])
    if which == 0:
        assert torch.all(torch.isnan(lse[:, hit]))
    else:
        assert torch.equal(lse, want_l)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens,h,hk", [
    ([1] * 64, [300 + 9 * i for i in range(64)], 8, 1), ([2] * 32, [900 + 17 * i for i in range(32)], 8, 1),
    ([5] * 8, [700 + 90 * i for i in range(8)], 32, 4)])
def test_outputs_are_no_longer_or_shorter_than_they_should_be(new, lens, h, hk, dtype, quant):
    """The factor c for which c times the fp64 result is nearest to O is 1: roundings of weights and
    outputs are as often up as down.  Each of the 32768 or more elements is off by up to 2 2^-9 of
    sqrt(mean O^2) (a weight's rounding to 9 bits and the output's to 8, both at most 2^-9; sums of many
    values grow as O does), so that the mean of independent ones stays below 2^-12, 11 of its standard
    deviations of at most 2^-8 / sqrt(32768)."""
    d = 128
    s = build(new, lens, h, hk, d, 64, dtype, quant, seed=20)
    o, _ = attend(s, causal=False)
    assert api.get_status() == 0
    along, square, at = 0.0, 0.0, 0
    for b, n in enumerate(new):
        k, v = (s["values"][i][b].cuda().transpose(0, 1).repeat_interleave(h // hk, 0) for i in range(2))
        x = s["q"][at:at + n].double().transpose(0, 1) @ k.transpose(1, 2) * d ** -0.5
        want = torch.softmax(x, -1) @ v
        along += ((o[at:at + n].double().transpose(0, 1) - want) * want).sum().item()
        square += (want * want).sum().item()
        at += n
    assert abs(along / square) <= 2.0 ** -12


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("new,lens", [([5, 2, 1], [2, 900, 0]), ([400, 90], [300, 20]), ([300, 1, 64], [250, 900, 3])])
def test_the_widest_window_is_none(new, lens, quant):
    """More new tokens than keys, so that some stand before the first position; a window that reaches
    past any cache hides nothing."""
    s = build(new, lens, 8, 2, 64, 32, BF, quant, seed=22)
    want, want_l = attend(s)
    check(s, want, want_l)
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 301, 10 ** 6):
        o, lse = attend(s, window=window)
        assert api.get_status() == 0
        assert torch.equal(o, want) and torch.equal(lse, want_l), window


def _many(kind):
    if kind == "tiles":                                                       # 160 rows and fewer, none
        new = [20 - i % 7 * 3 if i % 11 else 0 for i in range(140)]
        return new, [n + 37 * (i % 23) for i, n in enumerate(new)]
    if kind == "chunks apart":                                                # behind 32, 64, .. others and beside them
        new = [150] + [1] * 31 + [40] + [1] * 70 + [0] * 40 + [60, 1, 33] + [2] * 200 + [90]
    else:                                                                     # none at the ends
        new = [0] * 33 + [1] * 64 + [25] * 3 + [0] + [1] * 32 + [50] + [1] * 31 + [0] * 70
    return new, [n + (29 * i) % 400 for i, n in enumerate(new)]


@pytest.mark.parametrize("dtype,quant", [(BF, False), (BF, True), (FP, True)])
@pytest.mark.parametrize("kind", ["tiles", "chunks apart", "chunks inside"])
def test_hundreds_of_sequences(kind, dtype, quant):
    new, lens = _many(kind)
    s = build(new, lens, 8, 1 if kind == "tiles" else 2, 64, 16, dtype, quant, seed=23)
    o, lse = attend(s)
    torch.cuda.synchronize()
    assert api.get_status_site() == (0, 0)
    check(s, o, lse)


def test_single_tokens_between_chunks_cost_what_they_cost_behind_them():
    """2048 sequences of one token between two chunks, and the same behind both: the same work, so the
    shortest of 20 runs in turn differ by noise, far below the quarter allowed (stepping over the
    sequences between two of a CTA's chunks one at a time added half)."""
    hk, page, d, n = 8, 64, 64, 2048
    runs = []
    for order in ([0] + [2] * n + [1], [0, 1] + [2] * n):
        new, lens = ([(500, 500, 1)[i] for i in order], [(900, 900, 64)[i] for i in order])
        need = torch.tensor([-(-m // page) for m in lens])
        first = need.cumsum(0) - need
        table = (first[:, None] + torch.arange(int(need.max()))).to(torch.int32).cuda()     # past a length: anyone's
        pages = [torch.ones(int(need.sum()), hk, page, d, dtype=BF, device="cuda") for _ in "kv"]
        q = torch.ones(sum(new), 4 * hk, d, dtype=BF, device="cuda")
        args = (q, *pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets(new).cuda(), max(new))
        api.paged_attention(*args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = api.paged_attention(*args)
        runs.append((g, args, out, []))
    for _ in range(20):
        for g, _, _, times in runs:
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            g.replay()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
    assert api.get_status() == 0
    for _, _, (o, _), _ in runs:
        assert torch.all(o == 1.0)
    assert min(runs[0][3]) <= 1.25 * min(runs[1][3]), [min(r[3]) for r in runs]
