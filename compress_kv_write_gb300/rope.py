"""Frequencies for kvq_rope_table, on the host: the plain ones, and those of contexts longer than a model was trained on."""
from __future__ import annotations

import math

import torch


def rope_frequencies(rot, base=10000.0, *, factor=1.0, how="blend", original=4096, slow=1.0, fast=32.0):
    """float64 [rot / 2] radians a position, base ** (-2 i / rot), for a context `factor` times the `original` one:

    how="linear"  every frequency divided by the factor (positions squeezed into the original range)
    how="base"    the base grown to base * factor ** (rot / (rot - 2)): the slowest frequency is divided by the factor, the
                  fastest stays (rot > 2)
    how="blend"   what turns `fast` times or more within the original context stays, what turns `slow` times or less is
                  divided by the factor, in between the two are mixed, linearly in the pair's index, from the first border
                  rounded down (at least 0) to the second rounded up (at most rot - 1): the YaRN method
    """
    if rot < 2 or rot % 2 or not base > 0 or not factor >= 1:
        raise ValueError("rot must be even and positive, base positive and factor at least 1")
    if how not in ("linear", "base", "blend"):
        raise ValueError("how must be linear, base or blend")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if how == "base" and factor > 1:
        if rot == 2:
            raise ValueError("a single pair has no slowest and fastest frequency")
        base = base * factor ** (rot / (rot - 2))
    freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2 * i / rot)
    if factor == 1 or how == "base":
        return freq
    if how == "linear":
        return freq / factor
    if not (original > 0 and fast > slow > 0 and base > 1):
        raise ValueError("blend takes original > 0, fast > slow > 0 and base > 1")
    # the (fractional) index of the pair that turns `n` times within the original context
    at = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    if at(slow) <= 0:  # not even the fastest pair turns more than `slow` times
        return freq / factor
    first, last = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    mix = ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
    return freq * (1 - mix) + freq / factor * mix
