"""Rotary tables for kv_append: cos and sin of every position and pair, made
once in 64 bits and rounded to fp32.

The kernel only multiplies by the table, so every frequency rule lives here.
Long positions keep their accuracy: an fp32 product position * frequency is off
by up to half an ulp of the angle (0.008 rad at 131072 rad).
"""

from __future__ import annotations

import math

import torch


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original: int = 0, slow: float = 1.0,
                     fast: float = 32.0) -> torch.Tensor:
    """The rot_dim / 2 angular frequencies, fp64.

    scaling: None    base ** (-2 i / rot_dim);
    "linear"         every frequency divided by `factor` (positions interpolated);
    "base"           the base raised so that the slowest pair's wavelength grows by `factor`;
    "bands"          per pair: one that turns more than `fast` times over the
                     `original` context keeps its frequency, one that turns less
                     than `slow` times is divided by `factor`, and in between the
                     two are mixed linearly in the number of turns' logarithm."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be a positive even number")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("'base' scaling needs two pairs")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-i / rot_dim)
    if scaling in (None, "base"):
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        if original < 1 or not 0 < slow < fast:
            raise ValueError("'bands' needs the original context length and 0 < slow < fast")
        turns = original * f / (2 * math.pi)
        keep = ((turns.log() - math.log(slow)) / (math.log(fast) - math.log(slow))).clamp(0, 1)
        return f * keep + f / factor * (1 - keep)
    raise ValueError(f"unknown scaling {scaling!r}")


def rope_table(max_pos: int, frequencies: torch.Tensor, attention_factor: float = 1.0,
               device="cuda") -> torch.Tensor:
    """[max_pos, rot_dim / 2, 2] fp32 (cos, sin), both multiplied by attention_factor."""
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * frequencies.double().cpu()
    return (torch.stack([a.cos(), a.sin()], -1) * attention_factor).float().contiguous().to(device)
