"""Frequency tables of the rotary prologue (ret.rotary): host arithmetic in fp64, nothing else.

RetNet rotates by theta_i = base^(-i / (rot/2 - 1)), i = 0 .. rot/2 - 1, the base's exponents evenly
spaced from 0 to 1 inclusive ("retnet"); rotary position embeddings usually take base^(-2 i / rot)
("rope"). For contexts longer than the `length` a model was trained on, by a factor s:

  "linear"  every frequency divided by s (position interpolation);
  "ntk"     the base enlarged to base * s^(rot / (rot - 2)), which divides the lowest "rope"
            frequency by s and leaves the highest alone;
  "yarn"    by the number of turns n_i = length * theta_i / (2 pi) that a pair makes over the trained
            length: divided by s where n_i <= 1, kept where n_i >= 32, blended linearly in between;
            scores are sharpened by the amplitude 0.1 ln(s) + 1 (YaRN, arXiv:2309.00071, section 3).
"""
from __future__ import annotations

import math

import torch


def frequencies(rot: int, base: float = 10000.0, schedule: str = "rope", scaling: str | None = None,
                factor: float = 1.0, length: int | None = None, device=None):
    """(freqs [rot / 2] fp64 in radians per position, amplitude) for ret.rotary."""
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot must be positive and even, got {rot}")
    if not base > 0 or not factor >= 1:
        raise ValueError(f"base must be positive and factor at least 1, got {base} and {factor}")
    half = rot // 2
    i = torch.arange(half, dtype=torch.float64)
    if schedule not in ("rope", "retnet"):
        raise ValueError(f"unknown schedule {schedule!r}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk":
        if schedule != "rope" or rot <= 2:
            raise ValueError("ntk scaling is defined for the rope schedule with rot above 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot) if schedule == "rope" else base ** (-i / max(1, half - 1))
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if length is None or length <= 0:
            raise ValueError("yarn scaling needs the trained length")
        keep = ((length * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = (1.0 - keep) * f / factor + keep * f
        amplitude = 0.1 * math.log(factor) + 1.0
    return f.to(device) if device is not None else f, amplitude
