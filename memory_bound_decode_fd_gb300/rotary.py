"""Rotary frequencies in 64 bits, made once per model on the host: what ``rope`` and
``rope_append`` take as ``inv_freq`` and ``scale``.

Pair i of rot_dim / 2 turns by position * inv_freq[i], inv_freq[i] = base^(-2 i / rot_dim). For
contexts longer than the trained one the frequencies are stretched:

* ``"linear"``: every frequency divided by ``factor`` (positions interpolated).
* ``"banded"``: by wavelength. A pair that makes more than ``high`` turns over the trained context
  keeps its frequency, one that makes fewer than ``low`` is divided by ``factor``, and between the
  two the frequency is blended linearly in the number of turns.
* ``"ramp"``: the same idea with the blend linear in the pair's index, between the index whose
  pair makes ``high`` turns and the one whose pair makes ``low`` (rounded outwards), and with
  cosine and sine scaled by 0.1 ln(factor) + 1.
"""

from __future__ import annotations

import math

import torch

ROPE_SCALINGS = ("none", "linear", "banded", "ramp")


def rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  trained_context: int = 8192, low: float | None = None, high: float | None = None,
                  device=None) -> tuple[torch.Tensor, float]:
    """(inv_freq float64 [rot_dim / 2], scale) for ``rope`` and ``rope_append``.

    ``low`` and ``high`` are numbers of turns over ``trained_context`` (default 1 and 4 for
    "banded", 1 and 32 for "ramp").
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be above 1 and finite, got {base}")
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}, got {scaling!r}")
    if scaling != "none" and not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor must be at least 1 and finite, got {factor}")
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    scale = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling in ("banded", "ramp"):
        lo = 1.0 if low is None else float(low)
        hi = (4.0 if scaling == "banded" else 32.0) if high is None else float(high)
        if not (0.0 < lo < hi and trained_context > 0):
            raise ValueError("0 < low < high and a positive trained_context are wanted")
        if scaling == "banded":
            keep = [(trained_context * x / (2 * math.pi) - lo) / (hi - lo) for x in f]
        else:
            def pair_of(turns: float) -> float:  # the index whose pair makes so many turns
                return rot_dim * math.log(trained_context / (turns * 2 * math.pi)) / (2 * math.log(base))

            first = max(0.0, math.floor(pair_of(hi)))
            last = min(rot_dim - 1.0, math.ceil(pair_of(lo)))
            keep = [1.0 - (i - first) / max(last - first, 0.001) for i in range(len(f))]
            scale = 0.1 * math.log(factor) + 1.0
        keep = [min(1.0, max(0.0, s)) for s in keep]
        f = [x / factor * (1.0 - s) + x * s for x, s in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64, device=device), scale
