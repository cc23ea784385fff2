"""Frequencies of rotary positions, and the form in which the kernels take them.

A head's pair i turns by position * frequency[i] radians.  `rope_frequencies` gives the usual
frequencies, plain or scaled for contexts longer than those trained on; `rope_phases` turns any
frequencies into turns a position as 64-bit binary fractions, whose product with a position wraps
around modulo one turn and stays exact however far the position is.
"""
from __future__ import annotations

import math

import torch


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original_context: int = 0, fast: float = 32.0,
                     slow: float = 1.0):
    """(fp32 [rot_dim / 2] radians a position, factor on the turned dims).

    scaling None: base^(-2 i / rot_dim).  "linear": every frequency divided by `factor`.
    "base": the base grown so that the slowest pair slows down by `factor` and the fastest stays.
    "bands": pairs that turn more than `fast` times over `original_context` positions stay, those
    that turn less than `slow` times are divided by `factor`, those between blend linearly, and
    turned dims grow by 0.1 ln(factor) + 1 (the interpolation by parts of "YaRN: Efficient Context
    Window Extension", section 3)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim = {rot_dim}: an even number of dims turns")
    if factor < 1.0 or base <= 1.0:
        raise ValueError(f"factor = {factor} (at least 1), base = {base} (above 1)")
    if scaling == "base":
        if rot_dim == 2:
            raise ValueError("one pair has no base to grow")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    freq = base ** (-i / rot_dim)
    grow = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "bands":
        if original_context < 1 or fast <= slow:
            raise ValueError("bands needs original_context and fast > slow")
        turns = original_context * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq / factor * (1 - keep) + freq * keep
        grow = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling = {scaling!r} (None, linear, base or bands)")
    return freq.to(torch.float32), grow


def rope_phases(frequencies: torch.Tensor) -> torch.Tensor:
    """int64 [n]: frequencies (radians a position) as turns a position, in units of 2^-64 modulo
    one turn (the bits of an unsigned number), on the same device."""
    turns = torch.remainder(frequencies.to(torch.float64) / (2 * math.pi), 1.0)
    high = torch.floor(turns * 2.0**32)  # (powers of two: exact)
    low = torch.floor((turns * 2.0**32 - high) * 2.0**32)
    return (high.to(torch.int64) << 32) | low.to(torch.int64)
