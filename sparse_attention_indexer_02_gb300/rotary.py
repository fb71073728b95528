"""Rotary positions: a model's frequencies, made once on the host and kept on
the device in the form the rotation kernels read.

A pair i of the rotated part turns by f_i a position, f_i = base^(-2i/R) for R
rotated elements, changed for contexts longer than a model was trained on:

  linear   f_i / factor                      (positions pressed together)
  base     base * factor^(R / (R - 2))       (the slowest pair turns `factor` times
                                              slower, the fastest as before)
  parts    pairs that turn often over the original context stay, those that do
           not complete a turn are divided by factor, a ramp between: with
           r_i = original f_i / (2 pi) turns and g = clamp((r_i - low) / (high - low), 0, 1),
           f_i (g + (1 - g) / factor).  The ramp runs over the turns; a model whose ramp
           runs over the pairs' indexes i has other values between: give its `frequencies`

`magnitude` multiplies the cosines and sines (an attention temperature that some
scalings bring along, such as 0.1 ln(factor) + 1).
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import _abi

_LAYOUTS = {"half": _abi.ROTARY_HALF, "pairs": _abi.ROTARY_PAIRS}


def inv_freq(rot_dim: int, base: float = 10000.0, scaling: Optional[dict] = None) -> list:
    """The frequencies f_i in radians a position, i < rot_dim / 2 (Python floats).
    scaling: None, or dict(kind="linear" or "base", factor=...), or
    dict(kind="parts", factor=..., original=..., low=..., high=...)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    base = float(base)
    if not (base > 0 and math.isfinite(base)):
        raise ValueError("base must be finite and positive")
    s = dict(scaling) if scaling is not None else {}
    kind = s.pop("kind", None)
    want = {None: set(), "linear": {"factor"}, "base": {"factor"}, "parts": {"factor", "original", "low", "high"}}
    if kind not in want or set(s) != want[kind]:
        raise ValueError("scaling must be None or a dict of kind 'linear' or 'base' with factor, or of kind 'parts' "
                         "with factor, original, low and high")
    if not all(math.isfinite(v) for v in s.values()) or (kind and not s["factor"] > 0):
        raise ValueError("a scaling's values must be finite, its factor positive")
    if kind == "base":
        if rot_dim == 2:
            raise ValueError("the base scaling needs more than one pair")
        base *= s["factor"] ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if kind == "linear":
        f = [x / s["factor"] for x in f]
    elif kind == "parts":
        if not s["high"] > s["low"]:
            raise ValueError("a ramp's high must be above its low")
        g = [min(1.0, max(0.0, (s["original"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"]))) for x in f]
        f = [x * (k + (1.0 - k) / s["factor"]) for x, k in zip(f, g)]
    return f


class Rotary:
    """What torch_api.rotate_heads and rotate_store_kv need of a model's rotary
    positions.

    rot_dim: elements of a head that are rotated, from element `offset` on;
    layout: "half" (pairs i, i + rot_dim / 2) or "pairs" (2i, 2i + 1);
    frequencies as inv_freq above, or given (radians a position, rot_dim / 2 of
    them).  freqs holds them as turns in units of 2^-64, modulo 2^64."""

    def __init__(self, rot_dim: int, *, base: float = 10000.0, layout: str = "half", offset: int = 0,
                 scaling: Optional[dict] = None, magnitude: float = 1.0, frequencies: Optional[Sequence[float]] = None,
                 device="cuda"):
        if layout not in _LAYOUTS:
            raise ValueError("layout must be 'half' or 'pairs'")
        if frequencies is None:
            frequencies = inv_freq(rot_dim, base, scaling)
        elif scaling is not None:
            raise ValueError("frequencies are given as they are: no scaling beside them")
        frequencies = [float(f) for f in frequencies]
        if rot_dim < 2 or rot_dim % 2 or len(frequencies) != rot_dim // 2:
            raise ValueError("rot_dim must be even, with rot_dim / 2 frequencies")
        if not all(math.isfinite(f) for f in frequencies) or not math.isfinite(magnitude):
            raise ValueError("frequencies and magnitude must be finite")
        if offset != int(offset):
            raise ValueError("offset must be a whole number")
        self.rot_dim, self.layout, self.offset, self.magnitude = rot_dim, _LAYOUTS[layout], int(offset), float(magnitude)
        self.frequencies = frequencies
        turns = [int(round(math.ldexp(math.fmod(f / (2 * math.pi), 1.0), 64))) % (1 << 64) for f in frequencies]
        self.freqs = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
