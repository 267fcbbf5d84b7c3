"""Rotary frequencies and their long-context scalings (host side, fp64; no attention arithmetic).

Pair j of a head turns by ``position * inv_freq[j]`` radians, inv_freq[j] = base^(-2j / rotary_dim).
A model used past the length it was trained on scales them:

  linear  every frequency divided by ``scale`` (positions are interpolated)
  ntk     base raised to base * scale^(rotary_dim / (rotary_dim - 2)): the slowest frequency is
          divided by ``scale``, the fastest kept
  bands   by the turns r a pair makes over ``trained`` positions: kept for r >= high, divided by
          ``scale`` for r <= low, blended linearly in r between
  yarn    the same idea blended linearly in the pair's index, between the indices that make
          ``high`` and ``low`` turns (rounded outwards, kept within 0 and rotary_dim - 1: the end
          may lie behind the last pair), with the amplitude factor 0.1 ln(scale) + 1
          (YaRN: Efficient Context Window Extension of Large Language Models, 2023)
"""
from __future__ import annotations

import math

import torch

SCALINGS = (None, "linear", "ntk", "bands", "yarn")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, scale: float = 1.0,
                     trained: int | None = None, low: float = 1.0, high: float | None = None,
                     device: torch.device | str = "cuda"):
    """(inv_freq fp64 [rotary_dim / 2] on ``device``, amplitude factor) for ``api.rope``.

    ``high`` defaults to 4 turns for ``bands`` and 32 for ``yarn``; both need ``trained``."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and at least 2, got {rotary_dim}")
    if not (base > 1.0 and math.isfinite(base)) or not (scale >= 1.0 and math.isfinite(scale)):
        raise ValueError(f"base must exceed 1 and scale be at least 1, got {base}, {scale}")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}, got {scaling!r}")
    if scaling in ("bands", "yarn"):
        high = (4.0 if scaling == "bands" else 32.0) if high is None else float(high)
        if trained is None or trained < 1 or not 0.0 < low < high:
            raise ValueError(f"{scaling} needs trained >= 1 and 0 < low < high")
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("ntk needs at least two pairs")
        base = base * scale ** (rotary_dim / (rotary_dim - 2))
    j = torch.arange(rotary_dim // 2, dtype=torch.float64)
    freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * j / rotary_dim)
    factor = 1.0
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "bands":
        turns = trained * freq / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freq = keep * freq + (1.0 - keep) * freq / scale
    elif scaling == "yarn":
        def index(turns):  # the (fractional) pair that makes this many turns over `trained`
            return rotary_dim * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        first = max(math.floor(index(high)), 0)
        last = min(math.ceil(index(low)), rotary_dim - 1)
        ramp = ((j - first) / max(last - first, 0.001)).clamp(0.0, 1.0)
        freq = (1.0 - ramp) * freq + ramp * freq / scale
        factor = 0.1 * math.log(scale) + 1.0
    return freq.to(device), factor
