"""Paged caches for the tests: building one from contiguous keys and values, and the e4m3 row
quantisation written from its definition with integer arithmetic on numpy fp64."""
from __future__ import annotations

import numpy as np
import torch

# every finite e4m3 value >= 0 in ascending order: codes 0 .. 0x7E
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(0x7F)])


def quantise_rows(x: torch.Tensor):
    """(values, exponents) of rows [.., d] in fp64: each row's smallest e with max|finite| <= 448 2^e
    (clamped to the type's range) and the nearest e4m3 multiple of 2^e, ties to the even code, that
    the type can hold (240 * 2^8 for the largest fp16); NaN for what is not finite."""
    lo, hi = (-15, 8) if x.dtype == torch.float16 else (-126, 119)
    v = x.double().cpu().numpy()
    finite = np.isfinite(v)
    top = np.where(finite, np.abs(v), 0.0).max(-1, initial=0.0)
    e = np.full(top.shape, lo)
    while True:
        grow = (top > 448.0 * 2.0 ** e) & (e < hi)
        if not grow.any():
            break
        e = e + grow
    y = np.where(finite, np.abs(v), 0.0) / (2.0 ** e)[..., None]
    i = np.clip(np.searchsorted(E4M3, y, side="right") - 1, 0, len(E4M3) - 2)
    below, above = y - E4M3[i], E4M3[i + 1] - y
    up = (above < below) | ((above == below) & (i % 2 == 1))
    q = E4M3[np.where(up, i + 1, i)]
    if x.dtype == torch.float16:
        q = np.where((e == 8)[..., None], np.minimum(q, 240.0), q)
    q = q * (2.0 ** e)[..., None]
    return torch.from_numpy(np.where(finite, np.copysign(q, v), np.nan)), torch.from_numpy(e)


def page_tables(lens, page, g, spare=2, extra_columns=1):
    """(table int32 [B, max_pages], pages in the pool): every sequence gets pages of its own in a
    random order; unused entries hold -1."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1) + extra_columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def offsets(counts):
    return torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32)


def locate(table, b, pos, page):
    """(page numbers, slots) of positions `pos` (a tensor) of sequence b."""
    return table[b, pos // page].long(), pos % page
