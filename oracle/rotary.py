"""Oracle: the rotary embedding's other forms -- scaled frequencies, tables at any position, part of a head, pairs.

The forms are those of models whose rotation is not the rotate-half, base-10000 one of ``rope``; the pages have no
counterpart.  Angles are reduced exactly (whole-number arithmetic on the frequency's bits), so that a table entry at a
far position is the cosine of the true angle; the rotation rounds as ``rope_rotate`` does.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .rope import bf16_to_f32, f32_to_bf16_bits

# 2 pi to 200 bits, as a fraction
TWO_PI = Fraction(0x6487ED5110B4611A62633145C06E0E68948127044533E63A010, 1 << 200)


def frequencies(R: int, base: float = 10000.0, scaling: dict = None):
    """The scaled frequencies [R/2] and the amplitude, by the definitions of mixed_step.h."""
    kind = "plain" if scaling is None else scaling["kind"]
    if kind == "base":
        base = base * scaling["factor"] ** (R / (R - 2))
    out, amplitude = [], 1.0
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        if kind == "linear":
            f /= scaling["factor"]
        elif kind == "bands":
            turns = scaling["original_len"] * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - scaling["low"]) / (scaling["high"] - scaling["low"])))
            f = (1 - keep) * f / scaling["factor"] + keep * f
        elif kind == "ramp":
            # pair x turns original_len base^(-2x/R) / (2 pi) times
            x = [R / 2 * math.log(scaling["original_len"] / (2 * math.pi * t), base) for t in (scaling["high"], scaling["low"])]
            lo, hi = max(math.floor(x[0]), 0), min(math.ceil(x[1]), R - 1)
            stretch = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f = stretch * f / scaling["factor"] + (1 - stretch) * f
            amplitude = scaling.get("amplitude") or (0.1 * math.log(scaling["factor"]) + 1 if scaling["factor"] > 1 else 1.0)
        out.append(f)
    return np.array(out), amplitude


def table_entry(p: int, f: float, amplitude: float = 1.0):
    """(cos, sin) of the angle p f, reduced exactly, times the amplitude, in fp64."""
    turns = Fraction(float(f)) * int(p) / TWO_PI
    frac = float(turns - round(turns))
    return amplitude * math.cos(2 * math.pi * frac), amplitude * math.sin(2 * math.pi * frac)


def rotate(x_bits: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Rotate the first R = 2 cos.shape[1] elements of bf16 rows x [n, H, D] by per-row cos/sin; returns bf16 bits."""
    half = cos.shape[1]
    x = bf16_to_f32(x_bits)
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    c, s = cos[:, None, :].astype(np.float32), sin[:, None, :].astype(np.float32)
    out = np.array(x_bits, copy=True)
    out[..., a] = f32_to_bf16_bits(np.subtract(np.multiply(x[..., a], c), np.multiply(x[..., b], s)))
    out[..., b] = f32_to_bf16_bits(np.add(np.multiply(x[..., b], c), np.multiply(x[..., a], s)))
    return out
