"""Frequencies of rotary positions (the freqs and mscale of rope and rope_append), plain or scaled for contexts
longer than the one a model was trained on."""
import math

import torch


def rope_freqs(rot, base=10000.0, scaling=None, factor=1.0, trained_len=4096, slow_turns=1.0, fast_turns=32.0, device="cuda"):
    """(freqs float64 [rot/2], mscale): pair i turns by freqs[i] = base^(-2i/rot) radians a position.

    scaling None;
    "linear": positions interpolated, freqs / factor;
    "ntk": base * factor^(rot / (rot - 2)), which leaves the fastest pair as it is and slows the slowest by factor;
    "yarn": pairs that turn more than fast_turns times in trained_len positions stay, those below slow_turns are slowed by
    factor, a linear ramp over the turns between; mscale = 1 + 0.1 ln(factor) (YaRN, Peng et al. 2023)."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot}: expected an even number of at least 2")
    if factor < 1.0:
        raise ValueError(f"factor={factor} is below 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = trained_len * f / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        mscale = 1.0 + 0.1 * math.log(factor)
    return f.to(device), mscale
