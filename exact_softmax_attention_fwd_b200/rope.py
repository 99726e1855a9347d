"""Frequency tables of rotary positions (host side).

The kernels take the angles' frequencies as a table, ``inv_freq`` float64
[rotary_dim / 2] in radians per position, and a factor ``mscale`` on the cosines
and sines; this module makes the tables in use.  With n = rotary_dim / 2 and
base frequencies f_i = base^(-i/n):

* ``"none"``    f_i
* ``"linear"``  f_i / factor: positions squeezed into the trained range
* ``"base"``    the base stretched to base * factor^(n / (n - 1)), so that the
                fastest pair keeps its frequency and the slowest one is divided
                by exactly ``factor``
* ``"ramp"``    by how often a pair turns within ``original_length`` positions,
                r_i = original_length f_i / 2 pi: pairs with r_i >= fast_turns
                keep f_i, pairs with r_i <= slow_turns get f_i / factor, and the
                share of f_i falls linearly in r_i between the two; ``mscale``
                is 0.1 ln(factor) + 1.  Models trained with a ramp over the
                pair's index i instead (between bounds rounded to whole pairs)
                have other frequencies: pass their own table
"""
from __future__ import annotations

import math

KINDS = ("none", "linear", "base", "ramp")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_length: int = 8192, slow_turns: float = 1.0,
                     fast_turns: float = 32.0, device=None):
    """(inv_freq float64 [rotary_dim / 2] on ``device``, mscale) for attn_rope and
    attn_append_paged; see the module's notes for the scaling kinds."""
    import torch
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError("base must be over 1")
    if scaling not in KINDS:
        raise ValueError(f"scaling must be one of {KINDS}")
    if not factor >= 1.0 or not math.isfinite(factor):
        raise ValueError("factor must be at least 1")
    n = rotary_dim // 2
    i = torch.arange(n, dtype=torch.float64)
    mscale = 1.0
    if scaling == "base":
        if n < 2:
            raise ValueError("a stretched base needs two pairs at least")
        base = base * factor ** (n / (n - 1))
    freq = torch.exp(-i / n * math.log(base))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ramp":
        if original_length < 1 or not 0.0 <= slow_turns < fast_turns:
            raise ValueError("ramp needs original_length >= 1 and 0 <= slow_turns < fast_turns")
        turns = original_length * freq / (2.0 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return freq.to(device) if device is not None else freq, mscale
