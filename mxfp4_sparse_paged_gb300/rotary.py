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


# 1 / (2 pi) to 144 bits, 24 at a time: a product with half of an fp64 frequency is exact in fp64.
_TURNS = (10**49 << 144) // (2 * 31415926535897932384626433832795028841971693993751)
_TURNS = [_TURNS >> (24 * (5 - j)) & 0xFFFFFF for j in range(6)]


def rope_phases(frequencies: torch.Tensor) -> torch.Tensor:
    """int64 [n]: frequencies (radians a position) as turns a position, in units of 2^-64 modulo
    one turn (the bits of an unsigned number), right to a unit, on the same device."""
    f = frequencies.to(torch.float64)
    top = f.to(torch.float32).to(torch.float64)
    x = torch.stack([part * (digits * 2.0 ** (-24 * (j + 1)))  # of 24 and 29 bits
                     for j, digits in enumerate(_TURNS) for part in (top, f - top)])
    x = (x - x.trunc()) * 2.0**32
    high = x.floor()
    x = (x - high) * 2.0**32
    low = x.floor()
    rest = (x - low).sum(0).round().to(torch.int64)
    low = low.to(torch.int64).sum(0) + rest
    high = high.to(torch.int64).sum(0) + (low >> 32)
    return ((high + 2**31) % 2**32 - 2**31) * 2**32 + (low & 0xFFFFFFFF)
