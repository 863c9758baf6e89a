"""Rotary frequencies for long contexts, in fp64 on the host.

Plain rotary positions turn pair j of r rotated dims by position *
theta^(-2j/r). A model run past the context it was trained on slows the pairs
down, all alike or by wavelength; paged_rope_table_build_freqs takes the
frequencies this returns and builds the cos/sin table of every position.
"""
from __future__ import annotations

import math


def rope_frequencies(rope_theta: float, rot_dim: int = 64, scaling: str = "none", factor: float = 1.0,
                     original_context: int = 0, low: float = 1.0, high: float = 4.0,
                     ) -> tuple[list[float], float]:
    """The rot_dim / 2 inverse frequencies and the magnitude of cos and sin.

    scaling
      "none"    theta^(-2j/r)
      "linear"  positions interpolated: every frequency divided by factor
      "base"    the base raised to theta * factor^(r/(r-2)), so that the
                fastest pair keeps its speed and the slowest is divided by
                factor
      "banded"  by the turns t = original_context * f / 2 pi a pair makes over
                the original context: kept from `high` turns on, divided by
                factor up to `low` turns, between them f (k + (1 - k) /
                factor) with k = (t - low) / (high - low)
      "ramped"  as "banded" with the ramp linear in the pair's index between
                the indices (rounded outwards) that make `high` and `low`
                turns, and cos and sin multiplied by 0.1 ln(factor) + 1
    """
    if rot_dim < 8 or rot_dim > 64 or rot_dim % 8:
        raise ValueError("rot_dim must be 8, 16, .. 64")
    if not (rope_theta > 0 and math.isfinite(rope_theta)):
        raise ValueError("rope_theta must be positive and finite")
    if not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("factor must be at least 1")
    half = rot_dim // 2
    plain = [rope_theta ** (-2.0 * j / rot_dim) for j in range(half)]
    if scaling == "none":
        return plain, 1.0
    if scaling == "linear":
        return [f / factor for f in plain], 1.0
    if scaling == "base":
        theta = rope_theta * factor ** (rot_dim / (rot_dim - 2.0))
        return [theta ** (-2.0 * j / rot_dim) for j in range(half)], 1.0
    if scaling not in ("banded", "ramped"):
        raise ValueError(f"scaling {scaling!r} is not one of none, linear, base, banded, ramped")
    if original_context < 1 or not 0 < low < high:
        raise ValueError(f"{scaling} scaling needs original_context >= 1 and 0 < low < high")
    if scaling == "banded":
        keep = [(original_context * f / (2 * math.pi) - low) / (high - low) for f in plain]
        magnitude = 1.0
    else:
        if rope_theta <= 1:
            raise ValueError("ramped scaling needs rope_theta > 1")

        def index(turns: float) -> float:  # of the pair that makes `turns` turns
            return rot_dim * math.log(original_context / (2 * math.pi * turns)) / (2 * math.log(rope_theta))

        first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot_dim - 1)
        keep = [1.0 - (j - first) / max(last - first, 0.001) for j in range(half)]
        magnitude = 0.1 * math.log(factor) + 1.0
    keep = [min(max(k, 0.0), 1.0) for k in keep]
    return [f * k + f / factor * (1.0 - k) for f, k in zip(plain, keep)], magnitude
