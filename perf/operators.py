"""Rotary positions, the paged key/value cache and attention over it: what is measured.

Three operators that a serving or training step runs around exact attention, in the order a
step runs them:

* ``rope``: queries and keys are rotated by their positions; ``rope_bwd`` is its gradient.
* ``cache``: the new keys and values of every sequence are written to the pages of its cache
  (16-bit values, or e4m3 codes with one power-of-two scale per token and head), and a range
  of positions is read back as 16-bit values.
* ``paged``: the new tokens of every sequence (one, a few drafted ones, or a chunk of a prompt)
  attend to that sequence's pages.

Common layouts: tokens of all sequences end to end, ``[T, heads, d]``; sequence b owns the
tokens ``cu_q[b] .. cu_q[b + 1]``, which are the last positions of its ``seqlens[b]`` cached
ones; pages ``[P, H_kv, page, d]``; position p of sequence b lies in page
``page_table[b, p // page]`` at slot ``p % page``.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 16 sequences: launch latency is what counts
        _rope("rope_step_t16", tokens=16, heads=32, kv_heads=8, dim=128, rotary=128, dtype="bf16",
              interleaved=False, far=32768, factor=1.0, grad=False),
        # a training step's rotation and its gradient at the forward+backward workload's size
        _rope("rope_train_t16384_h16", tokens=16384, heads=16, kv_heads=16, dim=128, rotary=128, dtype="bf16",
              interleaved=True, far=8192, factor=1.0, grad=True),
        # an odd chunk of a long context: half of each head rotated, scaled amplitudes, fp16
        _rope("rope_chunk_t5001_partial", tokens=5001, heads=12, kv_heads=4, dim=64, rotary=32, dtype="fp16",
              interleaved=False, far=131072, factor=1.139, grad=False),
        # one token for each of 64 short sequences into an e4m3 cache
        _cache("cache_step_b64_e4m3", seqs=64, new=(1, 1), lens=(1, 4096), kv_heads=8, dim=128, page=16,
               dtype="bf16", quant=True, tail=True, plan=11),
        # whole prompts into a 16-bit cache and back, as when a sequence is moved
        _cache("cache_prompt_b4_n8192", seqs=4, new=(8192, 8192), lens=(8192, 8192), kv_heads=8, dim=128, page=64,
               dtype="bf16", quant=False, tail=False, plan=12),
        # ragged chunks into an e4m3 cache with odd head counts, everything read back
        _cache("cache_ragged_b7_e4m3_d64", seqs=7, new=(1, 3001), lens=(3001, 9001), kv_heads=5, dim=64, page=32,
               dtype="fp16", quant=True, tail=False, plan=13),
        # a small decoding step: latency
        _paged("paged_step_b4_small", seqs=4, chunks=0, new=(1, 1), lens=(200, 1000), heads=8, kv_heads=2, dim=64,
               page=16, dtype="bf16", quant=False, causal=True, window=-1, plan=21),
        # the decoding workload (16 sequences of 16K to 32K tokens) over pages
        _paged("paged_step_b16_32k", seqs=16, chunks=0, new=(1, 1), lens=(16384, 32768), heads=32, kv_heads=8,
               dim=128, page=64, dtype="bf16", quant=False, causal=True, window=-1, plan=22),
        # the same over an e4m3 cache
        _paged("paged_step_b16_32k_e4m3", seqs=16, chunks=0, new=(1, 1), lens=(16384, 32768), heads=32, kv_heads=8,
               dim=128, page=64, dtype="bf16", quant=True, causal=True, window=-1, plan=22),
        # five drafted tokens verified for each of 24 sequences, sliding window
        _paged("paged_verify_b24_window", seqs=24, chunks=0, new=(5, 5), lens=(700, 16384), heads=24, kv_heads=4,
               dim=128, page=32, dtype="fp16", quant=False, causal=True, window=4096, plan=23),
        # a chunk of 2048 prompt tokens at the end of a 32K context
        _paged("paged_chunk_n2048_32k", seqs=1, chunks=1, new=(2048, 2048), lens=(32768, 32768), heads=32, kv_heads=8,
               dim=128, page=64, dtype="bf16", quant=False, causal=True, window=-1, plan=24),
        # one odd chunk beside 16 decoding sequences, over an e4m3 cache
        _paged("paged_mixed_b17_e4m3", seqs=17, chunks=1, new=(1001, 1001), lens=(4001, 12001), heads=32, kv_heads=8,
               dim=128, page=16, dtype="bf16", quant=True, causal=True, window=-1, plan=25),
    ]


def _rope(name, **kw):
    return {"name": name, "op": "rope", **kw}


def _spans(kw):
    new, lens = kw.pop("new"), kw.pop("lens")
    return {**kw, "new_lo": new[0], "new_hi": new[1], "len_lo": lens[0], "len_hi": lens[1]}


def _cache(name, **kw):
    return {"name": name, "op": "cache", **_spans(kw)}


def _paged(name, **kw):
    return {"name": name, "op": "paged", **_spans(kw)}


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(2 ** rng.uniform(math.log2(lo), math.log2(hi))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "paged", "paged"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    plan = rng.randrange(1 << 30)
    if op == "rope":
        case = _rope("", tokens=_log(rng, 1, 16384), heads=min(32, kv_heads * group), kv_heads=kv_heads, dim=dim,
                     rotary=rng.choice([dim, dim // 2, dim // 4, dim - 10]), dtype=dtype,
                     interleaved=rng.random() < 0.5, far=_log(rng, 100, 131072),
                     factor=rng.choice([1.0, 1.139]), grad=rng.random() < 0.5)
    elif op == "cache":
        hi = _log(rng, 1, 4000)
        lo = _log(rng, hi, 9000)
        case = _cache("", seqs=_log(rng, 1, 7), new=(1, hi), lens=(lo, _log(rng, lo, 9001)),
                      kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, quant=rng.random() < 0.5,
                      tail=rng.random() < 0.5, plan=plan)
    else:
        window = rng.choice([-1, -1, 100, 4096])
        causal = window >= 0 or rng.random() < 0.8
        if rng.random() < 0.5:  # decoding, or a few drafted tokens
            new = rng.choice([1, 1, 2, 5, 7])
            lo = _log(rng, 8, 20000)
            case = _paged("", seqs=_log(rng, 1, 16), chunks=0, new=(1, new), lens=(lo, _log(rng, lo, 32768)),
                          heads=min(32 // kv_heads, group) * kv_heads, kv_heads=kv_heads, dim=dim, page=page,
                          dtype=dtype, quant=rng.random() < 0.5, causal=causal, window=window, plan=plan)
        else:  # chunks, alone or beside decoding sequences
            new = _log(rng, 8, 1500)
            lo = _log(rng, new, 8000)
            chunks = rng.choice([1, 1, 2])
            case = _paged("", seqs=chunks + rng.choice([0, 0, 5]), chunks=chunks, new=(max(1, new // 2), new),
                          lens=(lo, _log(rng, lo, 16384)), heads=min(32 // kv_heads, group) * kv_heads,
                          kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, quant=rng.random() < 0.5,
                          causal=causal, window=window, plan=plan)
    del case["name"]
    return case


def _plan(case):
    """(new tokens, cached lengths) of each sequence, from the case alone."""
    rng = random.Random(case["plan"])
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    if case["op"] == "paged" and case["chunks"]:  # the other sequences decode one token each
        new = [n if b < case["chunks"] else 1 for b, n in enumerate(new)]
    return [min(n, m) for n, m in zip(new, lens)], lens


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    dt = _TYPES[case["dtype"]]
    if case["op"] == "rope":
        t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        # queries and keys are slices of one fused projection's output
        qkv = torch.randn((t, h + 2 * hk, d), generator=g, device="cuda").to(dt)
        s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + hk]
        start = torch.randint(0, max(1, case["far"] - t + 1), (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(t, device="cuda")).to(torch.int32)
        j = torch.arange(case["rotary"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 10000.0 ** (-2.0 * j / case["rotary"])
        if case["grad"]:
            s["dq"] = torch.randn((t, h, d), generator=g, device="cuda").to(dt)
            s["dk"] = torch.randn((t, hk, d), generator=g, device="cuda").to(dt)
        return s
    new, lens = _plan(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(need) + 1), dtype=torch.int32, device="cuda")
    cols = torch.arange(table.shape[1], device="cuda")
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    used = cols[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[used] = order[(first[:, None] + cols[None, :])[used]]
    s["page_table"] = table
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    s["max_q"] = max(new)
    total = sum(new)
    shape = (pool, hk, page, d)
    for name in ("k", "v"):
        x = torch.randn(shape, generator=g, device="cuda").to(dt)
        s[name + "_scales"] = None
        if case["quant"]:
            codes, scales = _quantise(x.float(), dt)
            s[name + "_scales"] = scales.to(torch.float8_e8m0fnu)
            x = codes.to(torch.float8_e4m3fn)
        s[name + "_pages"] = x
    if case["op"] == "cache":
        qkv = torch.randn((total, 3 * hk, d), generator=g, device="cuda").to(dt)
        s["k"], s["v"] = qkv[:, hk:2 * hk], qkv[:, 2 * hk:]
        # read back: the new tokens alone, or everything
        s["starts"] = s["seqlens"] - torch.tensor(new, dtype=torch.int32, device="cuda") if case["tail"] else None
        back = new if case["tail"] else lens
        s["cu_k"] = torch.tensor([sum(back[:b]) for b in range(len(back) + 1)], dtype=torch.int32, device="cuda")
        s["total"] = sum(back)
    else:
        s["q"] = torch.randn((total, case["heads"], d), generator=g, device="cuda").to(dt)
        # the plain form computes sequences that bring about as many tokens together
        ones = [b for b in range(len(new)) if b >= case["chunks"]]
        s["together"] = ([ones] if ones else []) + [[b] for b in range(case["chunks"])]
        s["new"], s["lens"] = new, lens
    return s


def _quantise(x, dt):
    """(codes, scales) of the rows of x: the smallest power of two with |row| <= 448 scale."""
    m, e = torch.frexp(x.abs().amax(-1))               # amax = m 2^e, m in [1/2, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)                # 448 = 0.875 * 2^9
    e = e.clamp(-15, 8) if dt == torch.float16 else e.clamp(-126, 119)
    scale = torch.exp2(e.double()).float()
    return (x / scale[..., None]).to(torch.float8_e4m3fn).float(), scale


# ------------------------------------------------------------------ one pass
def run(s):
    return {"rope": _run_rope, "cache": _run_cache, "paged": _run_paged}[s["op"]](s)


def _run_rope(s):
    c = s["case"]
    kw = {"interleaved": c["interleaved"], "factor": c["factor"]}
    if own:
        from exact_io_aware_93_b200 import api
        out = api.rope(s["q"], s["k"], s["positions"], s["inv_freq"], **kw)
        if c["grad"]:
            out = out + api.rope_bwd(s["dq"], s["dk"], s["positions"], s["inv_freq"], **kw)
        return out
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    angle = torch.remainder(angle, 2 * math.pi).float()[:, None, :]
    cos, sin = angle.cos() * c["factor"], angle.sin() * c["factor"]
    out = (_rotate(s["q"], cos, sin, **kw), _rotate(s["k"], cos, sin, **kw))
    if c["grad"]:
        out = out + (_rotate(s["dq"], cos, -sin, **kw), _rotate(s["dk"], cos, -sin, **kw))
    return out


def _rotate(x, cos, sin, interleaved, factor):
    """Pairs (a, b) of the first columns become (a cos - b sin, b cos + a sin); the other columns
    keep their values."""
    n = 2 * cos.shape[-1]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:n:2], y[..., 1:n:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :n // 2], y[..., n // 2:n]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., n:]), -1).to(x.dtype)


def _slots(s, cu, first, total):
    """Of each of the `total` rows of a ragged batch: (page, slot) of its position, first[b] being
    the position of sequence b's first row."""
    rows = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    pos = first[b] + rows - cu[b]
    page = s["k_pages"].shape[2]
    return s["page_table"][b, pos // page].long(), pos % page


def _run_cache(s):
    c = s["case"]
    if own:
        from exact_io_aware_93_b200 import api
        api.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["seqlens"], s["cu_q"],
                         k_scales=s["k_scales"], v_scales=s["v_scales"])
        return api.cache_gather(s["k_pages"], s["v_pages"], s["page_table"], s["seqlens"], s["cu_k"], s["total"],
                                starts=s["starts"], k_scales=s["k_scales"], v_scales=s["v_scales"], dtype=s["k"].dtype)
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    to = _slots(s, s["cu_q"], s["seqlens"] - n, s["k"].shape[0])
    first = s["starts"] if s["starts"] is not None else torch.zeros_like(s["seqlens"])
    at = _slots(s, s["cu_k"], first, s["total"])
    return _write_and_read(s, "k", to, at, c), _write_and_read(s, "v", to, at, c)


def _write_and_read(s, name, to, at, c):
    x, pages, scales = s[name], s[name + "_pages"], s[name + "_scales"]
    if scales is None:
        pages[to[0], :, to[1]] = x
        return pages[at[0], :, at[1]]
    codes, scale = _quantise(x.float(), x.dtype)
    # indexing is not defined on the 8-bit types: the bytes are moved
    pages.view(torch.uint8)[to[0], :, to[1]] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    scales.view(torch.uint8)[to[0], :, to[1]] = scale.to(torch.float8_e8m0fnu).view(torch.uint8)
    codes = pages.view(torch.uint8)[at[0], :, at[1]].view(torch.float8_e4m3fn).float()
    scale = scales.view(torch.uint8)[at[0], :, at[1]].view(torch.float8_e8m0fnu).float()
    return (codes * scale[..., None]).to(x.dtype)


def _run_paged(s):
    c = s["case"]
    window = None if c["window"] < 0 else c["window"]
    if own:
        from exact_io_aware_93_b200 import api
        return api.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["seqlens"], s["cu_q"],
                                   s["max_q"], causal=c["causal"], window=window, k_scales=s["k_scales"],
                                   v_scales=s["v_scales"])
    out = torch.empty_like(s["q"])
    lse = torch.empty((c["heads"], s["q"].shape[0]), device="cuda")
    for seqs in s["together"]:
        _attend(s, seqs, out, lse)
    return out, lse


def _attend(s, seqs, out, lse):
    """Attention of the sequences `seqs`, padded to the longest of them."""
    c = s["case"]
    hk, d, page = c["kv_heads"], c["dim"], c["page"]
    group = c["heads"] // hk
    n = max(s["new"][b] for b in seqs)
    pages = -(-max(s["lens"][b] for b in seqs) // page)
    at = torch.tensor(seqs, device="cuda")
    table = s["page_table"][at, :pages].long()
    length = s["seqlens"][at].long()[:, None, None]
    count = (s["cu_q"][at + 1] - s["cu_q"][at]).long()
    row = torch.arange(n, device="cuda")
    live = row < count[:, None]                                       # [B, n]
    token = (s["cu_q"][at].long()[:, None] + row).clamp(max=s["q"].shape[0] - 1)
    pos = (length[:, :, 0] - count[:, None] + row)[:, :, None]        # [B, n, 1]
    key = torch.arange(pages * page, device="cuda")                   # [L]
    seen = key < length
    if c["causal"]:
        seen = seen & (key <= pos)
    if c["window"] >= 0:
        seen = seen & (key >= pos - c["window"])
    q = s["q"][token].float().view(len(seqs), n, hk, group, d)
    step = max(1, min(hk, (1 << 30) // (len(seqs) * n * group * pages * page)))  # heads at a time: the scores' memory
    for h in range(0, hk, step):
        k = _paged_values(s, "k", table, h, h + step)                 # [B, heads, L, d]
        v = _paged_values(s, "v", table, h, h + step)
        qh = q[:, :, h:h + step].permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, heads, n * group, d]
        x = torch.matmul(qh, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
        x = x.view(*x.shape[:2], n, group, -1).masked_fill(~seen[:, None, :, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top.clamp(min=-1e30))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:4], d) / total.clamp(min=1e-30)
        l = (top + torch.log(total))[..., 0]                          # [B, heads, n, group]
        o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)                    # [B, n, heads * group, d]
        l = l.permute(0, 2, 1, 3).flatten(2, 3)
        heads = slice(h * group, h * group + o.shape[2])
        out[token[live], heads] = o[live].to(out.dtype)
        lse[heads, token[live]] = l[live].t()


def _paged_values(s, name, table, lo, hi):
    pages, scales = s[name + "_pages"], s[name + "_scales"]
    if scales is None:
        x = pages[:, lo:hi][table].float()
    else:
        x = pages.view(torch.uint8)[:, lo:hi][table].view(torch.float8_e4m3fn).float()
        x = x * scales.view(torch.uint8)[:, lo:hi][table].view(torch.float8_e8m0fnu).float()[..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)                     # [B, pages, heads, page, d] -> [B, heads, L, d]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    h, hk, d = case.get("heads", 0), case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        passes = 2 if case["grad"] else 1
        elems = case["tokens"] * (h + hk) * d * passes
        turned = case["tokens"] * (h + hk) * case["rotary"] * passes
        return {"bytes": 4 * elems + passes * (4 * case["tokens"] + 4 * case["rotary"]), "flops": 3 * turned}
    new, lens = _plan(case)
    row = d + 1 if case["quant"] else 2 * d                           # bytes of one cached row
    table = 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "cache":
        back = new if case["tail"] else lens
        wrote = sum(new) * hk * 2 * (2 * d + row)                     # keys and values: read, written to the pages
        read = sum(back) * hk * 2 * (row + 2 * d)
        return {"bytes": wrote + read + table + 12 * len(lens), "flops": 0}
    pairs, keys = 0, 0
    for n, m in zip(new, lens):
        w = case["window"] if case["window"] >= 0 else m
        spans = [min(m - n + i, w) + 1 for i in range(n)] if case["causal"] else [m] * n
        pairs += sum(spans)
        keys += min(m, n + w) if case["causal"] else m
    moved = keys * hk * 2 * row + sum(new) * h * (2 * 2 * d + 4) + table + 12 * len(lens)
    return {"bytes": moved, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    new, lens = _plan(case)
    # flat index of every position of sequence b: page * slots + slot
    where = []
    for b, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        where.append(s["page_table"][b].long()[p // case["page"]] * case["page"] + p % case["page"])
    if case["op"] == "cache":
        return tuple(_exact_cache(s, case, name, new, lens, where) for name in ("k", "v"))
    return _exact_paged(s, case, new, lens, where)


def _exact_rope(s, case):
    half = case["rotary"] // 2
    if case["interleaved"]:
        first, second = torch.arange(half) * 2, torch.arange(half) * 2 + 1
    else:
        first, second = torch.arange(half), torch.arange(half) + half
    turn = torch.polar(torch.full((case["tokens"], half), case["factor"], dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * s["inv_freq"][None, :])

    def rotated(x, by):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * by[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = (rotated(s["q"], turn), rotated(s["k"], turn))
    if case["grad"]:
        out = out + (rotated(s["dq"], turn.conj()), rotated(s["dk"], turn.conj()))
    return out


def _rows64(s, name):
    """The cached rows [P * page, H_kv, d] in 64 bits."""
    x = s[name + "_pages"].to(torch.float32).double()
    if s[name + "_scales"] is not None:
        x = x * s[name + "_scales"].to(torch.float32).double().unsqueeze(-1)
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


def _exact_cache(s, case, name, new, lens, where):
    rows = _rows64(s, name)
    x = s[name].double()
    if case["quant"]:
        def two_to(e):  # built from its bits: a power function may be off in the last place
            return ((e.long() + 1023) << 52).view(torch.float64)

        # the smallest power of two that keeps the row within +-448, then the nearest value of
        # the 4-bit significand's grid (spacing 2^(exponent - 3), not below 2^-9), ties to even
        top = x.abs().amax(-1, keepdim=True)
        lo, hi = (-15, 8) if case["dtype"] == "fp16" else (-126, 119)
        power = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -300)))
        power = power - (top <= 224.0 * two_to(power)).double()       # where the logarithm fell just above
        power = (power + (top > 448.0 * two_to(power)).double()).clamp(lo, hi)
        y = x * two_to(-power)
        spacing = two_to((torch.frexp(y).exponent - 1).clamp(min=-6) - 3)
        x = torch.round(y / spacing) * spacing * two_to(power)
    at = 0
    out = []
    for b, (n, m) in enumerate(zip(new, lens)):
        rows[where[b][m - n:]] = x[at:at + n]
        at += n
        out.append(rows[where[b][m - n if case["tail"] else 0:]])
    return torch.cat(out)


def _exact_paged(s, case, new, lens, where):
    group = case["heads"] // case["kv_heads"]
    keys, values = _rows64(s, "k"), _rows64(s, "v")
    q = s["q"].double() / math.sqrt(case["dim"])
    out, lse, at = torch.zeros_like(q), torch.zeros(case["heads"], q.shape[0], dtype=torch.float64, device="cuda"), 0
    for b, (n, m) in enumerate(zip(new, lens)):
        t = torch.arange(m - n, m, device="cuda")[:, None]
        u = torch.arange(m, device="cuda")[None, :]
        hidden = torch.zeros((n, m), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= u > t
        if case["window"] >= 0:
            hidden |= u < t - case["window"]
        for h in range(case["heads"]):
            score = q[at:at + n, h] @ keys[where[b], h // group].T
            score[hidden] = -math.inf
            out[at:at + n, h] = torch.softmax(score, -1) @ values[where[b], h // group]
            lse[h, at:at + n] = torch.logsumexp(score, -1)
        at += n
    return out, lse
